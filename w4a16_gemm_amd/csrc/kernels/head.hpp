// Softmax cross entropy over a quantised vocabulary head, in pieces of the vocabulary:
//   l_v = W^_v x,  lse = log sum_v exp l_v,  loss = lse - l_target,
//   dx = dloss (sum_v c_v W^_v),  c_v = exp(l_v - lse) - [v == target].
// The logits of a tile of 64, 128 or 256 rows by 256 columns live in its accumulators and
// never leave the compute unit: the forward pass writes the maximum and the sum of
// exponentials of every row and column tile (8 bytes for 256 logits), which a second kernel
// joins; the backward pass computes the logits of a piece again, writes its c as binary16
// into a workspace and multiplies that with the piece's weights (transposed.hpp), pieces
// added in fp32.  Only rows with a target take part: the plan of plan.hpp with one expert.
//
// c is rounded to binary16 times 2^14: |c| <= 1 stays below 2^14, and down to 2^-28 it keeps
// the 11 bits of a normal number.  What the rounding of a row's largest entry, the target's,
// would do to the whole row is taken back: its remainder is added in fp32 at the end.
#pragma once

#include "experts.hpp"
#include "low.hpp"

namespace w4a16 {

constexpr float kCoeffLog2 = 14.f, kCoeffScale = 16384.f;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}

// Sum / maximum over the 16 lanes of a row of lanes, in every lane.
__device__ __forceinline__ float row16_sum(float v) {
  v += dpp<0xB1>(v);    // quad_perm [1, 0, 3, 2]
  v += dpp<0x4E>(v);    // quad_perm [2, 3, 0, 1]
  v += dpp<0x141>(v);   // row_half_mirror
  v += dpp<0x140>(v);   // row_mirror
  return v;
}
__device__ __forceinline__ float row16_max(float v) {
  v = fmaxf(v, dpp<0xB1>(v));
  v = fmaxf(v, dpp<0x4E>(v));
  v = fmaxf(v, dpp<0x141>(v));
  v = fmaxf(v, dpp<0x140>(v));
  return v;
}

// (maximum, sum of 2^(x log2 e - maximum log2 e)) of two sets of logits together.  An empty
// set has the maximum -infinity and the sum 0; a NaN stays in the sum.
struct MaxSum {
  float m, s;
};
__device__ __forceinline__ float exp_diff(float a, float b) { return __builtin_amdgcn_exp2f((a - b) * kLog2e); }
__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b) {
  const float m = fmaxf(a.m, b.m);
  const float base = m == -INFINITY ? 0.f : m;
  return {m, a.s * exp_diff(a.m, base) + b.s * exp_diff(b.m, base)};
}

struct HeadRows {
  const int32_t* target;   // [M]
  float* label;            // [places] forward: the target's logit; backward: the remainder of c
  const float* lse;        // [M] backward
};

// part [column tile][place]: forward; coeff [place][pitch]: backward, the columns from v0.
struct HeadOut {
  MaxSum* part;
  half_t* coeff;
  int pitch, v0, v1, vocab;
  size_t places;
};

// What a tile knows of its rows, in LDS.
struct HeadTileRows {
  int32_t* source;   // row of x
  int32_t* label;
  float* lse;        // backward
};

// c 2^14 of logits, as binary16, and the remainder of the target's c (backward).  All but the
// target's take one fma before the exponential: the rounding of lse log2 e is 2^-24 of that, as
// that of lse itself is, and below binary16's up to an lse of 2^13; the target's c may be small
// against its p and keeps the difference.
// (Two operations per coefficient less: the coefficients of a piece of 1229 rows 267 -> 244 us,
// of 8192 1033 -> 990 us.)
struct HeadCoeff {
  const HeadTileRows& own;
  const RowTile& tile;
  const HeadRows& rows;
  int n0, vocab;

  template <int COUNT>
  __device__ __forceinline__ void operator()(int row, int col, int step, const float (&v)[COUNT], half_t (&o)[COUNT]) const {
    const float lse = own.lse[row], base = __builtin_fmaf(lse, kLog2e, -kCoeffLog2);
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
      const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(v[i], kLog2e, -base));
      o[i] = static_cast<half_t>(n0 + col + step * i < vocab ? e : 0.f);
    }
    const int at = own.label[row] - n0 - col;   // step i: the target's is v[i]
    if (static_cast<uint32_t>(at) < static_cast<uint32_t>(step * COUNT) && at % step == 0) {
#pragma unroll
      for (int i = 0; i < COUNT; ++i)
        if (at == step * i) {
          const float c = exp_diff(v[i], lse) - 1.f;
          o[i] = static_cast<half_t>(c * kCoeffScale);
          if (row < tile.rows) rows.label[tile.first + row] = c - static_cast<float>(o[i]) * (1.f / kCoeffScale);
        }
    }
  }
};

template <int MB, int BITS, bool GRAD, int BM>
__device__ __forceinline__ void head_tile(const half_t* x, int x_rows, const Layers& l, unsigned char* smem,
                                          const HeadTileRows& own, const RowTile& tile, const HeadRows& rows,
                                          const HeadOut& to, int n0, int ct) {
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const TileLoader<4, MB, BITS, BM> ld(x, x_rows, l, smem, own.source, tile.rows, n0, tid, wave);
  float4_t acc[MB][4];
  tile_product(ld, l.zeros, smem, tid, wave, acc);
  __syncthreads();   // the ring's memory is used again
  const int lane = tid & 63, wm = wave >> 2, wn = wave & 3, lr = lane & 15, lq = lane >> 4;
  if constexpr (!GRAD) {
    const int c0 = n0 + wn * 64 + lr;   // this lane's column of block 0
    const bool whole = n0 + 256 <= to.vocab;
    MaxSum* red = reinterpret_cast<MaxSum*>(smem);   // [wn][row]
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = wm * 16 * MB + 16 * mb + 4 * lq + r;
        const int at = own.label[row] - c0;   // 16 nb: the target's logit is this lane's
        float v[4], m = -INFINITY;
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
          v[nb] = whole || c0 + 16 * nb < to.vocab ? acc[mb][nb][r] : -INFINITY;
          m = fmaxf(m, v[nb]);
        }
        if (at >= 0 && at < 64 && at % 16 == 0 && row < tile.rows)
          rows.label[tile.first + row] = at < 32 ? (at < 16 ? v[0] : v[1]) : (at < 48 ? v[2] : v[3]);
        m = row16_max(m);
        const float base = m == -INFINITY ? 0.f : m;
        float s = 0.f;
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) s += exp_diff(v[nb], base);
        s = row16_sum(s);
        if (lr == 0) red[wn * BM + row] = {m, s};
      }
    __syncthreads();
    if (tid < tile.rows)
      to.part[static_cast<size_t>(ct) * to.places + tile.first + tid] =
          join(join(red[tid], red[BM + tid]), join(red[2 * BM + tid], red[3 * BM + tid]));
  } else {
    store_tile<4, MB>(
        acc, smem, tid, HeadCoeff{own, tile, rows, n0, to.vocab},
        [&](int row, int col, half8_t v) {
          if (row < tile.rows && n0 + col < to.v1)
            *reinterpret_cast<half8_t*>(to.coeff + static_cast<size_t>(tile.first + row) * to.pitch + n0 + col - to.v0) = v;
        });
  }
}

// Logits of the rows of the plan's tiles against the columns [v0, v1), 256 at a time.
template <int BITS, bool GRAD, int BM>
__global__ __launch_bounds__(512, BM == 256 ? 2 : 4) void head_kernel(const half_t* __restrict__ x, int x_rows, int gathered, Layers layers,
                                                   SlotPlan plan, HeadRows rows, HeadOut to) {
  extern __shared__ __align__(16) unsigned char smem[];
  const int tid = threadIdx.x;
  RowTile tile;
  int ct;
  if (!find_tile(plan, (to.v1 - to.v0 + 255) / 256, blockIdx.x, tile, ct)) return;
  int32_t* words = reinterpret_cast<int32_t*>(smem + tile_lds<BITS, BM>() - 16 * BM);
  const HeadTileRows own{words, words + BM, reinterpret_cast<float*>(words + 2 * BM)};
  if (tid < tile.height) {
    const int place = tile.first + min(tid, tile.rows - 1), m = plan.order[place];
    own.source[tid] = gathered ? place : m;
    own.label[tid] = rows.target[m];
    if (GRAD) own.lse[tid] = rows.lse[m];
  }
  __syncthreads();
  const int n0 = to.v0 + 256 * ct;
  if (BM == 256 && tile.height == 256)
    head_tile<BM == 256 ? 8 : 4, BITS, GRAD, BM>(x, x_rows, layers, smem, own, tile, rows, to, n0, ct);
  else if (tile.height == 128)
    head_tile<4, BITS, GRAD, BM>(x, x_rows, layers, smem, own, tile, rows, to, n0, ct);
  else
    head_tile<2, BITS, GRAD, BM>(x, x_rows, layers, smem, own, tile, rows, to, n0, ct);
}

// The order of up to 64 rows by their targets, as the plan's: rows with a target first.  By
// the first wavefront of a workgroup, into LDS; returns the number of rows with a target.
__device__ __forceinline__ int order_rows(const int32_t* target, int M, int vocab, int lane, int32_t* order) {
  const int t = lane < M ? target[lane] : -1;
  const unsigned long long with = __ballot(t >= 0 && t < vocab);
  const int valid = __popcll(with), before = __popcll(with & ((1ull << lane) - 1));
  order[with >> lane & 1 ? before : valid + lane - before] = lane;
  return valid;
}

// The same on tiles of up to 64 rows (low.hpp).
template <int RB, int BITS, bool GRAD>
__device__ __forceinline__ void head_low_tile(const half_t* x, int x_rows, const Layers& l, unsigned char* smem,
                                              const HeadTileRows& own, const RowTile& tile, const HeadRows& rows,
                                              const HeadOut& to, int n0, int ct) {
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const LowLoader<BITS> ld(x, x_rows, l, smem, own.source, tile.rows, n0, tid, wave);
  LowSums<RB> acc;
  low_product(ld, l.zeros, smem, tid, wave, acc);
  __syncthreads();   // the ring's memory is used again
  const int lane = tid & 63, lc = lane & 31, lh = lane >> 5;
  if constexpr (!GRAD) {
    // The logits turn in LDS, 4 bytes of padding per row of 256, so that a wavefront has whole
    // rows, 4 columns per lane: two reductions over a wavefront per row of the tile that is
    // there, where the accumulators' layout takes one per row and 32 columns (37 rows: 66 -> 56 us).
    constexpr int PITCH = 260;
    float* turn = reinterpret_cast<float*>(smem);
    static_assert(64 * PITCH * 4 <= low_lds<BITS>() - kLowRowsLds, "fits the ring");
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        turn[(32 * b + 8 * (r >> 2) + 4 * lh + (r & 3)) * PITCH + 32 * wave + lc] = acc.b[b][r];
    __syncthreads();
    const int col = n0 + 4 * lane;
    for (int row = wave; row < tile.rows; row += 8) {
      const float4_t l4 = *reinterpret_cast<const float4_t*>(turn + row * PITCH + 4 * lane);
      float v[4], m = -INFINITY;
      const int at = own.label[row] - col;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = col + i < to.vocab ? l4[i] : -INFINITY;
        m = fmaxf(m, v[i]);
        if (at == i) rows.label[tile.first + row] = v[i];
      }
      m = row16_max(m);
      m = fmaxf(m, __shfl_xor(m, 16));
      m = fmaxf(m, __shfl_xor(m, 32));
      const float base = m == -INFINITY ? 0.f : m;
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) s += exp_diff(v[i], base);
      s = row16_sum(s);
      s += __shfl_xor(s, 16);
      s += __shfl_xor(s, 32);
      if (lane == 0) to.part[static_cast<size_t>(ct) * to.places + tile.first + row] = {m, s};
    }
  } else {
    store_low<RB>(
        acc, smem, tid, HeadCoeff{own, tile, rows, n0, to.vocab},
        [&](int row, int col, half8_t v) {
          if (row < tile.rows && n0 + col < to.v1)
            *reinterpret_cast<half8_t*>(to.coeff + static_cast<size_t>(tile.first + row) * to.pitch + n0 + col - to.v0) = v;
        });
  }
}

// plan.counts NULL: up to 64 rows without a plan, each workgroup orders them itself.
template <int BITS, bool GRAD>
__global__ __launch_bounds__(512, 4) void head_low_kernel(const half_t* __restrict__ x, int x_rows, int gathered,
                                                          Layers layers, SlotPlan plan, HeadRows rows, HeadOut to) {
  extern __shared__ __align__(16) unsigned char smem[];
  const int tid = threadIdx.x;
  int32_t* words = reinterpret_cast<int32_t*>(smem + low_lds<BITS>() - kLowRowsLds);
  const HeadTileRows own{words, words + 64, reinterpret_cast<float*>(words + 128)};
  RowTile tile;
  int ct;
  if (plan.counts) {
    if (!find_tile(plan, (to.v1 - to.v0 + 255) / 256, blockIdx.x, tile, ct)) return;
    if (tid < 64) {
      const int place = tile.first + min(tid, tile.rows - 1), m = plan.order[place];
      own.source[tid] = gathered ? place : m;
      own.label[tid] = rows.target[m];
      if (GRAD) own.lse[tid] = rows.lse[m];
    }
    __syncthreads();
  } else {
    ct = blockIdx.x;
    if (ct * 256 >= to.v1 - to.v0) return;
    if (tid < 64) {
      const int valid = order_rows(rows.target, x_rows, to.vocab, tid, own.source);
      if (tid == 0) words[192] = valid;
    }
    __syncthreads();
    tile = {};
    tile.rows = words[192];
    if (tile.rows == 0) return;
    if (tid < tile.rows) own.label[tid] = rows.target[own.source[tid]];
    __syncthreads();
  }
  const int n0 = to.v0 + 256 * ct;
  if (tile.rows > 32)
    head_low_tile<2, BITS, GRAD>(x, x_rows, layers, smem, own, tile, rows, to, n0, ct);
  else
    head_low_tile<1, BITS, GRAD>(x, x_rows, layers, smem, own, tile, rows, to, n0, ct);
}

// Joins the column tiles of 16 places per workgroup, 64 of them side by side in a fixed
// order; rows without a target get zeros.
__global__ __launch_bounds__(1024) void head_join_kernel(const MaxSum* __restrict__ part, int tiles, size_t places,
                                                         SlotPlan plan, const int32_t* __restrict__ target, int vocab,
                                                         const float* __restrict__ label, int M,
                                                         float* __restrict__ loss, float* __restrict__ lse) {
  __shared__ MaxSum red[64][16];
  __shared__ int32_t few[65];   // without a plan: the order, and the rows with a target
  const int at = threadIdx.x & 15, group = threadIdx.x >> 4;
  if (!plan.counts) {
    if (threadIdx.x < 64) {
      const int valid = order_rows(target, M, vocab, threadIdx.x, few);
      if (threadIdx.x == 0) few[64] = valid;
    }
    __syncthreads();
  }
  const int p = blockIdx.x * 16 + at, valid = plan.counts ? plan.counts[1] : few[64];
  MaxSum a = {-INFINITY, 0.f};
  if (p < valid) {
    int t = group;
    for (; t + 3 * 64 < tiles; t += 4 * 64) {
      MaxSum v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = part[static_cast<size_t>(t + 64 * i) * places + p];
      a = join(a, join(join(v[0], v[1]), join(v[2], v[3])));
    }
    for (; t < tiles; t += 64) a = join(a, part[static_cast<size_t>(t) * places + p]);
  }
  red[group][at] = a;
  __syncthreads();
  for (int step = 32; step > 0; step >>= 1) {
    if (group < step) red[group][at] = join(red[group][at], red[group + step][at]);
    __syncthreads();
  }
  if (group != 0 || p >= M) return;
  const int m = plan.counts ? plan.order[p] : few[p];
  if (p >= valid) {
    loss[m] = 0.f;
    lse[m] = 0.f;
    return;
  }
  a = red[0][at];
  const float v = a.m + __builtin_amdgcn_logf(a.s) * kLn2;
  lse[m] = v;
  loss[m] = v - label[p];
}

// dx[m] = dloss[m] (sum of the parts 2^-14 + remainder W^_target), rounded once; zeros for
// rows without a target.  One workgroup per place, eight channels per thread.
template <int BITS>
__global__ __launch_bounds__(256) void head_dx_kernel(const float* __restrict__ part, size_t places, int most, int side, int outputs,
                                                      SlotPlan plan, Layers l, const int32_t* __restrict__ inverse,
                                                      const int32_t* __restrict__ target,
                                                      const float* __restrict__ remainder,
                                                      const float* __restrict__ dloss, half_t* __restrict__ dx) {
  const int p = blockIdx.x, K = l.K;
  const size_t m = plan.order[p];
  const bool valid = p < plan.counts[1];
  const int cols = (K + 255) / 256;
  const int label = valid ? target[m] : 0;
  const float rest = valid ? remainder[p] : 0.f, d = valid ? dloss[m] : 0.f;
  const int tile = valid ? plan.tile_of[m] : 0;
  const Pieces rule(max(1, plan.counts[0] * cols), most, side, outputs);
  constexpr int PER = 32 / BITS;   // channels per word
  const uint32_t* codes = l.qw + static_cast<size_t>(label) * (K / PER);
  auto consts = [&](int k) {
    const int g = k >> l.gshift;
    return make_consts(load_zero<BITS>(l.zeros, g, l.N, label), l.scales[static_cast<size_t>(g) * l.N + label]);
  };
  for (int k0 = 8 * threadIdx.x; k0 < K; k0 += 8 * 256) {
    half8_t o{};
    if (valid) {
      const RowTile row = plan.tiles[tile];
      float s[8] = {}, w[8];
      if (inverse) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int k = min(static_cast<uint32_t>(inverse[k0 + i]), static_cast<uint32_t>(K - 1));
          const int pieces = rule.of(row, tile, k / 256, cols);
          for (int q = 0; q < pieces; ++q) s[i] += part[(q * places + p) * K + k];
          if constexpr (BITS == 4)
            w[i] = static_cast<float>(dequant_word(codes[k / 8], consts(k))[k % 8]);
          else
            w[i] = static_cast<float>(dequant_word8(codes[k / 4], consts(k))[k % 4]);
        }
      } else {
        const int pieces = rule.of(row, tile, k0 / 256, cols);
        for (int q = 0; q < pieces; ++q) {
          const float* at = part + (q * places + p) * K + k0;
          const float4_t lo = *reinterpret_cast<const float4_t*>(at), hi = *reinterpret_cast<const float4_t*>(at + 4);
#pragma unroll
          for (int i = 0; i < 4; ++i) s[i] += lo[i], s[4 + i] += hi[i];
        }
        const DequantConsts c = consts(k0);
        if constexpr (BITS == 4) {
          const half8_t v = dequant_word(codes[k0 / 8], c);
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = static_cast<float>(v[i]);
        } else {
          const half4_t lo = dequant_word8(codes[k0 / 4], c), hi = dequant_word8(codes[k0 / 4 + 1], c);
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = static_cast<float>(lo[i]), w[4 + i] = static_cast<float>(hi[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = static_cast<half_t>(d * (s[i] * (1.f / kCoeffScale) + rest * w[i]));
    }
    *reinterpret_cast<half8_t*>(dx + m * K + k0) = o;
  }
}

}  // namespace w4a16
