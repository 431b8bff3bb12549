// Softmax cross entropy over a quantised vocabulary head, in pieces of the vocabulary:
//   l_v = W^_v x,  lse = log sum_v exp l_v,  loss = lse - l_target,
//   dx = dloss (sum_v c_v W^_v),  c_v = exp(l_v - lse) - [v == target].
// The logits of a 256-row by 256-column tile live in the accumulators of the large tile and
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

namespace w4a16 {

constexpr float kCoeffScale = 16384.f;
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

template <int MB, int BITS, bool GRAD>
__device__ __forceinline__ void head_tile(const half_t* x, int x_rows, const Layers& l, unsigned char* smem,
                                          const int32_t* source, const int32_t* row_of, const RowTile& tile,
                                          const HeadRows& rows, const HeadOut& to, int n0, int ct) {
  constexpr int BM = 32 * MB;
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const auto ld = rows_loader<4, MB, BITS>(x, x_rows, l, smem, source, tile.rows, n0, l.N, tid, wave);
  float4_t acc[MB][4];
  big_tile_product<4, MB, BITS>(ld, l.zeros, smem, l.K, l.gshift, tid, wave, 1, acc);
  const int lane = tid & 63, wm = wave >> 2, wn = wave & 3, lr = lane & 15, lq = lane >> 4;
  const int c0 = n0 + wn * 64 + lr;   // this lane's column of block 0
  if constexpr (!GRAD) {
    __syncthreads();   // the ring's memory is used again
    MaxSum* red = reinterpret_cast<MaxSum*>(smem);   // [wn][row]
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = wm * 16 * MB + 16 * mb + 4 * lq + r;
        const int label = rows.target[row_of[min(row, tile.rows - 1)]];
        float v[4], m = -INFINITY;
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
          v[nb] = c0 + 16 * nb < to.vocab ? acc[mb][nb][r] : -INFINITY;
          if (c0 + 16 * nb == label && row < tile.rows) rows.label[tile.first + row] = v[nb];
          m = fmaxf(m, v[nb]);
        }
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
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = wm * 16 * MB + 16 * mb + 4 * lq + r;
        if (row >= tile.rows) continue;
        const int m = row_of[row];
        const int label = rows.target[m];
        const float lse = rows.lse[m];
        half_t* out = to.coeff + static_cast<size_t>(tile.first + row) * to.pitch - to.v0;
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
          const int col = c0 + 16 * nb;
          if (col >= to.v1) continue;
          float c = col < to.vocab ? exp_diff(acc[mb][nb][r], lse) : 0.f;
          if (col == label) c -= 1.f;
          const half_t h = static_cast<half_t>(c * kCoeffScale);
          if (col == label) rows.label[tile.first + row] = c - static_cast<float>(h) * (1.f / kCoeffScale);
          out[col] = h;
        }
      }
  }
}

// Logits of the rows of the plan's tiles against the columns [v0, v1), 256 at a time.
template <int BITS, bool GRAD>
__global__ __launch_bounds__(512) void head_kernel(const half_t* __restrict__ x, int x_rows, int gathered, Layers layers,
                                                   SlotPlan plan, HeadRows rows, HeadOut to) {
  extern __shared__ __align__(16) unsigned char smem[];
  const int tid = threadIdx.x;
  RowTile tile;
  int ct;
  if (!find_tile(plan, (to.v1 - to.v0 + 255) / 256, blockIdx.x, tile, ct)) return;
  int32_t* m = reinterpret_cast<int32_t*>(smem + experts_lds<BITS>() - kTileRowsLds);
  int32_t* source = m + kBigBM;
  if (tid < tile.rows) {
    m[tid] = plan.order[tile.first + tid];
    source[tid] = gathered ? tile.first + tid : m[tid];
  }
  __syncthreads();
  const int n0 = to.v0 + 256 * ct;
  if (tile.height == 256)
    head_tile<8, BITS, GRAD>(x, x_rows, layers, smem, source, m, tile, rows, to, n0, ct);
  else if (tile.height == 128)
    head_tile<4, BITS, GRAD>(x, x_rows, layers, smem, source, m, tile, rows, to, n0, ct);
  else
    head_tile<2, BITS, GRAD>(x, x_rows, layers, smem, source, m, tile, rows, to, n0, ct);
}

// Joins the column tiles of 64 places per workgroup, 16 of them side by side in a fixed
// order; rows without a target get zeros.
__global__ __launch_bounds__(1024) void head_join_kernel(const MaxSum* __restrict__ part, int tiles, size_t places,
                                                         SlotPlan plan, const float* __restrict__ label, int M,
                                                         float* __restrict__ loss, float* __restrict__ lse) {
  __shared__ MaxSum red[16][64];
  const int lane = threadIdx.x & 63, group = threadIdx.x >> 6;
  const int p = blockIdx.x * 64 + lane, valid = plan.counts[1];
  MaxSum a = {-INFINITY, 0.f};
  if (p < valid)
    for (int t = group; t < tiles; t += 16) a = join(a, part[static_cast<size_t>(t) * places + p]);
  red[group][lane] = a;
  __syncthreads();
  if (group != 0 || p >= M) return;
  const int m = plan.order[p];
  if (p >= valid) {
    loss[m] = 0.f;
    lse[m] = 0.f;
    return;
  }
  for (int g = 1; g < 16; ++g) a = join(a, red[g][lane]);
  const float v = a.m + __builtin_amdgcn_logf(a.s) * kLn2;
  lse[m] = v;
  loss[m] = v - label[p];
}

// dx[m] = dloss[m] (sum of the parts 2^-14 + remainder W^_target), rounded once; zeros for
// rows without a target.  One workgroup per place.
template <int BITS>
__global__ __launch_bounds__(256) void head_dx_kernel(const float* __restrict__ part, size_t places, int splits,
                                                      SlotPlan plan, Layers l, const int32_t* __restrict__ inverse,
                                                      const int32_t* __restrict__ target,
                                                      const float* __restrict__ remainder,
                                                      const float* __restrict__ dloss, half_t* __restrict__ dx) {
  const int p = blockIdx.x, K = l.K;
  const size_t m = plan.order[p];
  const bool valid = p < plan.counts[1];
  const int label = valid ? target[m] : 0;
  const float rest = valid ? remainder[p] : 0.f, d = valid ? dloss[m] : 0.f;
  for (int k0 = 8 * threadIdx.x; k0 < K; k0 += 8 * 256) {
    half8_t o{};
    if (valid) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t k = k0 + i;
        if (inverse) k = min(static_cast<uint32_t>(inverse[k]), static_cast<uint32_t>(K - 1));
        float s = 0.f;
        for (int q = 0; q < splits; ++q) s += part[(q * places + p) * K + k];
        const int g = k >> l.gshift;
        const DequantConsts c = make_consts(load_zero<BITS>(l.zeros, g, l.N, label), l.scales[static_cast<size_t>(g) * l.N + label]);
        float w;
        if constexpr (BITS == 4)
          w = static_cast<float>(dequant_word(l.qw[static_cast<size_t>(label) * (K / 8) + k / 8], c)[k % 8]);
        else
          w = static_cast<float>(dequant_word8(l.qw[static_cast<size_t>(label) * (K / 4) + k / 4], c)[k % 4]);
        o[i] = static_cast<half_t>(d * (s * (1.f / kCoeffScale) + rest * w));
      }
    }
    *reinterpret_cast<half8_t*>(dx + m * K + k0) = o;
  }
}

}  // namespace w4a16
