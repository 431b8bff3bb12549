// Low-rank adapters of many requests beside a shared projection, and their gradients.
//
// Row m of the activations belongs to adapter i = index[m].  Forward:
//   h[m] = A_i x[m]                                  (shrink, K -> R)
//   out[m] = y[m] + s_i B_i h[m]                     (expand, R -> N)
// Backward:
//   g[m] = B_i^T dy[m]                               (shrink, N -> R, B transposed first)
//   dx[m] = dx0[m] + s_i A_i^T g[m]                  (expand, R -> K)
//   dB_i = s_i sum_m dy[m] h[m]^T,  dA_i = s_i sum_m g[m] x[m]^T       (outer)
//
// All of them are tall products with one side of R <= 128, on v_mfma_f32_16x16x32_f16
// with fp32 sums.  Every operand that comes from memory is binary16 and enters exactly; h
// and g are fp32 sums and enter as two binary16 terms (hi + lo, 22 bits) after a division
// by a power of two that brings the largest of them to [2^13, 2^14), so nothing overflows
// and the split loses less than the fp32 sums do.
//
// Rows are worked on in tiles of 16 MT rows of one adapter each; rows of one adapter are
// found through a row plan (below), so any order of rows costs the same products.
#pragma once

#include "act8.hpp"

namespace w4a16 {

// How rows are grouped by adapter.  Class of a row: its adapter, or L ("none") for an
// index outside [0, L).
//   index == NULL             every row belongs to adapter 0
//   off == NULL (M <= 64)     each wavefront groups the rows itself, one row per lane
//   else                      off[c] = first sorted position of class c (L + 2 entries),
//                             perm[p] = row at sorted position p (plan_rows_kernel)
struct RowPlan {
  const int32_t* index;
  const int32_t* off;
  const int32_t* perm;
  int M, L;
};

constexpr int kInlineRows = 64;

__device__ __forceinline__ int row_class(int i, int L) { return i >= 0 && i < L ? i : L; }

// Stable grouping by class: workgroup c counts the rows of smaller classes, then places
// its own rows in order.  No atomics, so the order (and with it every sum) is fixed.
__global__ __launch_bounds__(1024) void plan_rows_kernel(const int32_t* __restrict__ index, int M, int L,
                                                         int32_t* __restrict__ off, int32_t* __restrict__ perm) {
  __shared__ int part[16];
  const int c = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int below = 0;
  for (int m = tid; m < M; m += 1024) below += row_class(index[m], L) < c ? 1 : 0;
  for (int d = 1; d < 64; d <<= 1) below += __shfl_xor(below, d);
  if (lane == 0) part[wave] = below;
  __syncthreads();
  int at = 0;
  for (int w = 0; w < 16; ++w) at += part[w];
  if (tid == 0) {
    off[c] = at;
    if (c == L) off[L + 1] = M;
  }
  for (int m0 = 0; m0 < M; m0 += 1024) {
    const int m = m0 + tid;
    const bool mine = m < M && row_class(index[m], L) == c;
    const uint64_t b = __ballot(mine);
    __syncthreads();   // the previous round's (first: the counts') reads of part are done
    if (lane == 0) part[wave] = __popcll(b);
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < 16; ++w) {
      before += w < wave ? part[w] : 0;
      total += part[w];
    }
    if (mine) perm[at + before + __popcll(b & ((1ull << lane) - 1ull))] = m;
    at += total;
  }
}

// Number of tile slots for T rows per tile (host and device agree on it): slots of class
// c start at off[c] / T + c, which leaves room for every class's last partial tile.
__host__ __device__ inline int tile_slots(const RowPlan& p, int T) {
  if (!p.index) return (p.M + T - 1) / T;
  const int most = p.M / T + p.L + 1;
  return !p.off && p.M < most ? p.M : most;
}

struct Tile {
  int adapter;   // L: rows without an adapter
  int count;     // rows in the tile, 0: empty slot
};

// Tile of a slot; every thread of the workgroup calls it, `rows` (LDS, T entries) holds
// the tile's rows afterwards, entries past the count repeating a valid row.
template <int T>
__device__ __forceinline__ Tile find_tile(const RowPlan& p, int slot, int32_t* rows) {
  const int tid = threadIdx.x, lane = tid & 63;
  Tile t;
  if (!p.index) {
    const int first = slot * T;
    t.adapter = 0;
    t.count = min(T, p.M - first);
    if (tid < T) rows[tid] = first + min(tid, t.count - 1);
  } else if (p.off) {
    int n = 0;
    for (int c0 = 0; c0 <= p.L; c0 += 64) {
      const int c = c0 + lane;
      const uint64_t b = __ballot(c <= p.L && p.off[min(c, p.L)] / T + c <= slot);
      n += __popcll(b);
      if (b != ~0ull) break;
    }
    const int c = n - 1;   // class 0 starts at slot 0, so n >= 1
    const int lo = p.off[c], hi = p.off[c + 1];
    const int first = lo + (slot - (lo / T + c)) * T;
    t.adapter = c;
    t.count = max(0, min(T, hi - first));
    if (tid < T && t.count > 0) rows[tid] = p.perm[first + min(tid, t.count - 1)];
  } else {
    const int cls = lane < p.M ? row_class(p.index[min(lane, p.M - 1)], p.L) : -1;
    int rank = 0;   // among the earlier rows of the same class
    for (int k = 0; k < p.M; ++k) rank += (__shfl(cls, k) == cls && k < lane) ? 1 : 0;
    uint64_t starts = __ballot(lane < p.M && rank % T == 0);
    for (int k = 0; k < slot; ++k) starts &= starts - 1;
    t.adapter = p.L;
    t.count = 0;
    if (starts != 0) {
      const int s = __builtin_ctzll(starts);
      t.adapter = __shfl(cls, s);
      const int r0 = __shfl(rank, s);
      const bool mine = lane < p.M && cls == t.adapter && rank >= r0 && rank < r0 + T;
      t.count = __popcll(__ballot(mine));
      if (tid < 64) {
        if (mine) rows[rank - r0] = lane;
        if (lane >= t.count && lane < T) rows[lane] = s;
      }
    }
  }
  t.adapter = __builtin_amdgcn_readfirstlane(t.adapter);
  t.count = __builtin_amdgcn_readfirstlane(t.count);
  __syncthreads();
  return t;
}

__device__ __forceinline__ float finite_magnitude(float v) {
  const float a = __builtin_fabsf(v);
  return a <= 3.402823466e38f ? a : 0.0f;
}

// Exponent e with m < 2^e (m > 0), 0 for m == 0.
__device__ __forceinline__ int top_exponent(float m) { return m > 0.0f ? __builtin_amdgcn_frexp_expf(m) : 0; }

// v = h 2^shift as hi + lo in binary16.  An infinite or NaN h keeps it in hi alone.
__device__ __forceinline__ void split_half(float h, int shift, half_t& hi, half_t& lo) {
  const float v = __builtin_ldexpf(h, shift);
  hi = static_cast<half_t>(v);
  const float r = v - static_cast<float>(hi);
  lo = static_cast<half_t>(__builtin_fabsf(v) <= 65504.0f ? r : 0.0f);
}

constexpr int kSplitTop = 14;   // split operands are below 2^14
constexpr int kNoExponent = -1000;   // of values that are all zero

// --- shrink: out[s][m][j] = sum over the channels of slice s of x[m][c] w[i][j][c] -------
//
// x [M][C], w [L][R][C], C % 8 == 0.  A wavefront holds 16 MT rows x 16 NT ranks of sums
// and walks steps of 32 channels, both operands as they lie in memory (lane (r, q): row r,
// channels 8 q .. 8 q + 7 of the step).  The wavefronts of a workgroup take turns along
// the slice; their sums are added in LDS in a fixed order.  A row's result depends on its
// own x alone, so the rows repeated to fill a tile are computed and not stored.
template <int NT, int MT, int W>
__global__ __launch_bounds__(64 * W) void lora_shrink_kernel(const half_t* __restrict__ x, const half_t* __restrict__ w,
                                                             RowPlan plan, int C, int R, float* __restrict__ out) {
  constexpr int T = 16 * MT;
  constexpr int U = NT * MT >= 8 ? 2 : 4;   // steps whose loads are in flight together
  __shared__ int32_t rows[T];
  __shared__ float4_t red[(W / 2 > 0 ? W / 2 : 1) * MT * NT * 64];
  const int S = gridDim.y, s = blockIdx.y;
  const Tile tile = find_tile<T>(plan, blockIdx.x, rows);
  if (tile.count == 0) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lq = lane >> 4;
  float* o = out + static_cast<size_t>(s) * plan.M * R;
  if (tile.adapter == plan.L) {
    for (int i = tid; i < tile.count * R; i += 64 * W) o[static_cast<size_t>(rows[i / R]) * R + i % R] = 0.0f;
    return;
  }
  const half_t* xr[MT];
  const half_t* wr[NT];
#pragma unroll
  for (int a = 0; a < MT; ++a) xr[a] = x + static_cast<size_t>(rows[16 * a + lr]) * C;
#pragma unroll
  for (int t = 0; t < NT; ++t)
    wr[t] = w + (static_cast<size_t>(tile.adapter) * R + min(16 * t + lr, R - 1)) * C;
  float4_t acc[MT][NT] = {};
  const int steps = (C + 31) >> 5;
  const int b = static_cast<int>(static_cast<int64_t>(steps) * s / S);
  const int e = static_cast<int>(static_cast<int64_t>(steps) * (s + 1) / S);
  for (int st = b + wave * U; st < e; st += W * U) {
    half8_t xa[U][MT], wb[U][NT];
    if (st + U <= e && (st + U) * 32 <= C) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = (st + u) * 32 + 8 * lq;
#pragma unroll
        for (int a = 0; a < MT; ++a) xa[u][a] = *reinterpret_cast<const half8_t*>(xr[a] + c);
#pragma unroll
        for (int t = 0; t < NT; ++t) wb[u][t] = *reinterpret_cast<const half8_t*>(wr[t] + c);
      }
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = (st + u) * 32 + 8 * lq;
        const bool in = st + u < e && c < C;   // channels outside are zero on both sides
        const int cc = min(c, C - 8);
#pragma unroll
        for (int a = 0; a < MT; ++a) {
          const half8_t v = *reinterpret_cast<const half8_t*>(xr[a] + cc);
          xa[u][a] = in ? v : half8_t{};
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const half8_t v = *reinterpret_cast<const half8_t*>(wr[t] + cc);
          wb[u][t] = in ? v : half8_t{};
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int t = 0; t < NT; ++t)
          acc[a][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(xa[u][a], wb[u][t], acc[a][t], 0, 0, 0);
  }
#pragma unroll
  for (int half = W / 2; half > 0; half >>= 1) {
    if (wave >= half && wave < 2 * half)
#pragma unroll
      for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int t = 0; t < NT; ++t) red[((wave - half) * MT * NT + a * NT + t) * 64 + lane] = acc[a][t];
    __syncthreads();
    if (wave < half)
#pragma unroll
      for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[a][t] += red[(wave * MT * NT + a * NT + t) * 64 + lane];
    __syncthreads();
  }
  if (wave != 0) return;
#pragma unroll
  for (int a = 0; a < MT; ++a)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 16 * a + 4 * lq + r, j = 16 * t + lr;
        if (i < tile.count && j < R) o[static_cast<size_t>(rows[i]) * R + j] = acc[a][t][r];
      }
}

// --- expand: out[m][c] = binary16(base[m][c] + s_i sum_j h[m][j] w_i[c][j]) ---------------
//
// h = sum of S slices [S][M][R].  TRANS == false: w [L][C][R]; TRANS: w [L][R][C].
// A workgroup of 4 wavefronts takes 16 MT rows x 512 channels.  Each wavefront keeps the
// weights of its 128 channels in registers (8 MFMA tiles of 16 channels as the A operand)
// and walks the rows 16 at a time (the B operand, from LDS, where the workgroup put the
// split h once); base of the next 16 rows is in flight meanwhile.  HBM-bound: 2 bytes
// read and 2 written per element.
// The channels are dealt to the MFMA rows so that a lane ends up with four runs of 8
// consecutive channels of one row (run u at 32 u + 8 q), and base and out move as 16-byte
// accesses, 64 bytes of a row per quarter wavefront.  !TRANS: MFMA row 4 q + r of tile t
// is channel 32 (t / 2) + 8 q + 4 (t % 2) + r.  TRANS: lane (r, q) loads octet (r >> 2) + 4
// (r & 3) of its 8 ranks and transposes the 8 x 8 block in registers; tile t has channel t
// of every octet, and MFMA row 4 q + r is octet q + 4 r.
// R <= 16 (PACKED): hi and lo share one MFMA, ranks 0..15 of hi in its first 16 slots and
// of lo in the last 16, against the same weights.  Larger R: F fragments of 32 ranks,
// one MFMA for hi and one for lo each.
// base may equal out (every element is read and written by the same lane); rows without
// an adapter are copied, bit for bit.  h_out (not NULL): the workgroups of the first
// channels write the summed h.

// The 8 x 8 block of binary16 values in v (one row per register quad) by columns: element
// i of column t is element t of row i.
__device__ __forceinline__ half8_t column8(const uint4 (&v)[8], int t) {
  const uint32_t sel = (t & 1) ? 0x07060302u : 0x05040100u;
  uint32_t d[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 &u0 = v[2 * i], &u1 = v[2 * i + 1];
    const uint32_t e0 = t < 2 ? u0.x : t < 4 ? u0.y : t < 6 ? u0.z : u0.w;
    const uint32_t e1 = t < 2 ? u1.x : t < 4 ? u1.y : t < 6 ? u1.z : u1.w;
    d[i] = __builtin_amdgcn_perm(e1, e0, sel);
  }
  return __builtin_bit_cast(half8_t, (u32x4_t{d[0], d[1], d[2], d[3]}));
}

// Sum over the S slices of 8 consecutive floats, 4 slices in flight at a time.
__device__ __forceinline__ void sum_slices8(const float* __restrict__ p, size_t slice, int S, float (&v)[8]) {
  float4_t a = {}, b = {};
  for (int s0 = 0; s0 < S; s0 += 4) {
    float4_t x[4], y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float* q = p + min(s0 + k, S - 1) * slice;
      x[k] = *reinterpret_cast<const float4_t*>(q);
      y[k] = *reinterpret_cast<const float4_t*>(q + 4);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (s0 + k < S) {
        a += x[k];
        b += y[k];
      }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = a[j];
    v[4 + j] = b[j];
  }
}

template <int F, bool PACKED, int MT, bool TRANS>
__global__ __launch_bounds__(256) void lora_expand_kernel(const float* __restrict__ h, int S,
                                                          const half_t* __restrict__ w,
                                                          const float* __restrict__ scaling, RowPlan plan,
                                                          const half_t* base, half_t* out, float* __restrict__ h_out,
                                                          int C, int R) {
  constexpr int T = 16 * MT;
  constexpr int kBlock = 512;   // channels per workgroup: 4 wavefronts x 128
  constexpr int P = PACKED ? 1 : 2;
  __shared__ int32_t rows[T];
  __shared__ float factor[T];
  __shared__ half8_t split[MT][F][P][64];
  const Tile tile = find_tile<T>(plan, blockIdx.x, rows);
  if (tile.count == 0) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lq = lane >> 4;
  const int c_lo = blockIdx.y * kBlock;
  if (tile.adapter == plan.L) {
    if (base != out) {
      const int chunks = min(kBlock, C - c_lo) / 8;
      for (int i = tid; i < tile.count * chunks; i += 256) {
        const size_t at = static_cast<size_t>(rows[i / chunks]) * C + c_lo + 8 * (i % chunks);
        uint4 v = {0, 0, 0, 0};
        if (base) v = *reinterpret_cast<const uint4*>(base + at);
        *reinterpret_cast<uint4*>(out + at) = v;
      }
    }
    if (h_out && blockIdx.y == 0)
      for (int i = tid; i < tile.count * R; i += 256) h_out[static_cast<size_t>(rows[i / R]) * R + i % R] = 0.0f;
    return;
  }
  const int nm = (tile.count + 15) >> 4;   // groups of 16 rows
  const int c0 = c_lo + wave * 128;
  const int jq = PACKED ? (lq & 1) * 8 : lq * 8;

  // base of 16 rows, from the first group before anything else
  auto load_base = [&](int a, uint4 (&y)[4]) {
    const bool in = base && 16 * a + lr < tile.count;
    const half_t* p = base + static_cast<size_t>(rows[16 * a + lr]) * C;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = c0 + 32 * u + 8 * lq;
      y[u] = uint4{0, 0, 0, 0};
      if (in && c < C) y[u] = *reinterpret_cast<const uint4*>(p + c);
    }
  };
  uint4 y[4];
  load_base(0, y);

  // weights of 128 channels
  half8_t wf[F][8];
  const half_t* wl = w + static_cast<size_t>(tile.adapter) * R * C;
  if (c0 < C) {
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const int j0 = 32 * f + jq;
      const bool in = j0 < R;
      if constexpr (!TRANS) {
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          const int c = min(c0 + 32 * (t >> 1) + 8 * (lr >> 2) + 4 * (t & 1) + (lr & 3), C - 1);
          const half8_t v = *reinterpret_cast<const half8_t*>(wl + static_cast<size_t>(c) * R + (in ? j0 : 0));
          wf[f][t] = in ? v : half8_t{};
        }
      } else {
        const int cc = min(c0 + 8 * ((lr >> 2) + 4 * (lr & 3)), C - 8);
        uint4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = *reinterpret_cast<const uint4*>(wl + static_cast<size_t>(in ? j0 + i : i) * C + cc);
          if (!in) v[i] = uint4{0, 0, 0, 0};
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) wf[f][t] = column8(v, t);
      }
    }
  }

  // split h: wavefront w takes rows 16 a + lr for a = w, w + 4, ...
  const float si = scaling ? scaling[tile.adapter] : 1.0f;
  const size_t slice = static_cast<size_t>(plan.M) * R;
  for (int a = wave; a < nm; a += 4) {
    const size_t row = static_cast<size_t>(rows[16 * a + lr]) * R;
    float v[F][8];
    float top = 0.0f;
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const int j0 = 32 * f + jq;
      const bool in = j0 < R;
      sum_slices8(h + row + (in ? j0 : 0), slice, S, v[f]);
      if (h_out && blockIdx.y == 0 && in && 16 * a + lr < tile.count && (!PACKED || lq < 2)) {
        *reinterpret_cast<float4_t*>(h_out + row + j0) = float4_t{v[f][0], v[f][1], v[f][2], v[f][3]};
        *reinterpret_cast<float4_t*>(h_out + row + j0 + 4) = float4_t{v[f][4], v[f][5], v[f][6], v[f][7]};
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[f][j] = in ? v[f][j] : 0.0f;
        top = fmaxf(top, finite_magnitude(v[f][j]));
      }
    }
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    const int shift = kSplitTop - top_exponent(top);
    if (lq == 0) factor[16 * a + lr] = __builtin_ldexpf(si, -shift);
#pragma unroll
    for (int f = 0; f < F; ++f) {
      half8_t hi, lo;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        half_t vh, vl;
        split_half(v[f][j], shift, vh, vl);
        hi[j] = PACKED && lq >= 2 ? vl : vh;
        lo[j] = vl;
      }
      split[a][f][0][lane] = hi;
      if constexpr (!PACKED) split[a][f][P - 1][lane] = lo;
    }
  }
  __syncthreads();
  if (c0 >= C) return;

  for (int a = 0; a < nm; ++a) {
    uint4 next[4];
    if (a + 1 < nm) load_base(a + 1, next);
    float4_t acc[8] = {};
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const half8_t hf = split[a][f][p][lane];
#pragma unroll
        for (int t = 0; t < 8; ++t) acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(wf[f][t], hf, acc[t], 0, 0, 0);
      }
    if (16 * a + lr < tile.count) {
      const float fa = factor[16 * a + lr];
      half_t* po = out + static_cast<size_t>(rows[16 * a + lr]) * C;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int c = c0 + 32 * u + 8 * lq;
        const half8_t yv = __builtin_bit_cast(half8_t, y[u]);
        half8_t o;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float v = TRANS ? acc[i][u] : acc[2 * u + (i >> 2)][i & 3];
          o[i] = static_cast<half_t>(fmaf(v, fa, static_cast<float>(yv[i])));
        }
        if (c < C) *reinterpret_cast<half8_t*>(po + c) = o;
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) y[u] = next[u];
  }
}

// --- transpose: b [L][N][R] -> bt [L][R][N], the layout the shrink reads ------------------
constexpr int kTransposeRows = 128;

__global__ __launch_bounds__(256) void lora_transpose_kernel(const half_t* __restrict__ b, half_t* __restrict__ bt,
                                                             int N, int R) {
  extern __shared__ __align__(16) half_t tile[];   // [kTransposeRows][R + 2]
  const int n0 = blockIdx.x * kTransposeRows, nr = min(kTransposeRows, N - n0);
  const half_t* src = b + (static_cast<size_t>(blockIdx.y) * N + n0) * R;
  half_t* dst = bt + static_cast<size_t>(blockIdx.y) * R * N + n0;
  const int ld = R + 2;
  for (int i = threadIdx.x; i < nr * R / 8; i += 256) {
    const half8_t v = *reinterpret_cast<const half8_t*>(src + 8 * i);
    const int n = 8 * i / R, j = 8 * i % R;
#pragma unroll
    for (int e = 0; e < 8; ++e) tile[n * ld + j + e] = v[e];
  }
  __syncthreads();
  const int oct = nr / 8;   // N % 8 == 0
  for (int i = threadIdx.x; i < R * oct; i += 256) {
    const int j = i / oct, n = 8 * (i % oct);
    half8_t v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = tile[(n + e) * ld + j];
    *reinterpret_cast<half8_t*>(dst + static_cast<size_t>(j) * N + n) = v;
  }
}

// --- split: h (or the sum of S slices of g) as MFMA operands of the outer products --------
//
// One workgroup per slot of 32 rows of one adapter.  Fragment t of a slot holds ranks 16 t
// .. + 15: lane (r, q) has rank 16 t + r of rows 8 q .. 8 q + 7, first the hi terms of all
// lanes (1 KB), then the lo terms, in units of 2^exps[slot].  Rows past the slot's count
// and ranks past R are zero.  Done once per call instead of by every workgroup of 128
// channels that reads h.  blockIdx.y == 0 splits h (one slice), 1 splits g.
struct SplitTask {
  const float* h;
  int S;
  half_t* frags;     // [slots][NT][2][64][8]
  int32_t* exps;     // [slots]
};

constexpr int kSlotRows = 32;

__global__ __launch_bounds__(256) void lora_split_kernel(SplitTask t0, SplitTask t1, RowPlan plan, int R) {
  __shared__ int32_t rows[kSlotRows];
  __shared__ float tops[4];
  const SplitTask task = blockIdx.y == 0 ? t0 : t1;
  const int slot = blockIdx.x;
  const Tile tile = find_tile<kSlotRows>(plan, slot, rows);
  if (tile.count == 0 || tile.adapter == plan.L) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lr = lane & 15, lq = lane >> 4;
  const int NT = (R + 15) >> 4;
  const size_t slice = static_cast<size_t>(plan.M) * R;
  float v[2][8];   // at most 8 fragments: two per wavefront
  float top = 0.0f;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int j = 16 * (wave + 4 * k) + lr;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[k][i] = 0.0f;
    if (16 * (wave + 4 * k) >= R) continue;
    for (int s = 0; s < task.S; ++s)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[k][i] += task.h[s * slice + static_cast<size_t>(rows[8 * lq + i]) * R + min(j, R - 1)];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (j >= R || 8 * lq + i >= tile.count) v[k][i] = 0.0f;
      top = fmaxf(top, finite_magnitude(v[k][i]));
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
  if (lane == 0) tops[wave] = top;
  __syncthreads();
  top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
  const int e = top > 0.0f ? top_exponent(top) - kSplitTop : kNoExponent;
  if (tid == 0) task.exps[slot] = e;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int t = wave + 4 * k;
    if (t >= NT) continue;
    half8_t hi, lo;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      half_t a, b;
      split_half(v[k][i], e == kNoExponent ? 0 : -e, a, b);
      hi[i] = a;
      lo[i] = b;
    }
    half8_t* o = reinterpret_cast<half8_t*>(task.frags) + (static_cast<size_t>(slot) * NT + t) * 128 + lane;
    o[0] = hi;
    o[64] = lo;
  }
}

// --- outer: grad_i[c][j] = s_i sum over the rows of adapter i of x[m][c] h[m][j] ----------
//
// A wavefront sums 128 channels x 16 NT ranks over slots of 32 rows; the wavefronts of a
// workgroup take turns along the slots and are added in LDS in a fixed order.  Lane (r, q)
// loads 8 channels (octet r) of its 8 rows (8 q ..) and transposes the 8 x 8 block in
// registers, so that x goes from memory to the MFMA operand without LDS; the next slot's
// rows are in flight meanwhile.  The split h comes as ready operands.
// Every slot has a power of two of its own; the sums are kept in units of the largest seen
// (as the running maximum of a softmax is): a larger one rescales the sums, a smaller one
// the operands.  A slot's missing rows repeat its first one against zero operands.
// Q8: x is an 8-bit checkpoint, expanded after the transpose (which then moves bytes).
// CMAJOR: gradient [L][C][R] (channels are MFMA rows), else [L][R][C].
template <int NT, bool Q8>
struct OuterSlot {
  uint4 v[8];              // 8 rows of 8 channels (Q8: the codes in x and y)
  uint32_t s2[Q8 ? 4 : 1]; // scales of rows 2 i, 2 i + 1
  half8_t h[NT][2];        // hi and lo operands
  int e;                   // their power of two
};

// D slots in flight per wavefront.
template <int NT, int W, int D, bool Q8, bool CMAJOR>
__global__ __launch_bounds__(64 * W) void lora_outer_kernel(const half_t* __restrict__ x,
                                                            const uint8_t* __restrict__ codes,
                                                            const half_t* __restrict__ xs, int gshift,
                                                            const half_t* __restrict__ frags,
                                                            const int32_t* __restrict__ exps,
                                                            const float* __restrict__ scaling, RowPlan plan,
                                                            float* __restrict__ grad, int C, int R) {
  __shared__ float4_t red[W * NT * 64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lq = lane >> 4;
  const int c0 = blockIdx.x * 128;
  const int t0 = blockIdx.y * NT;
  const int ad = blockIdx.z;
  const int NTT = (R + 15) >> 4;   // fragments per slot
  // slots of the adapter: [first_slot, first_slot + n); positions lo .. hi - 1
  const int lo = plan.index ? plan.off[ad] : 0;
  const int hi = plan.index ? plan.off[ad + 1] : plan.M;
  const int first_slot = plan.index ? lo / kSlotRows + ad : 0;
  const int n = (hi - lo + kSlotRows - 1) / kSlotRows;
  const int cc = min(c0 + 8 * lr, C - 8);
  const int G = Q8 ? C >> gshift : 0;

  // Rows of slot k (clamped to the last slot: a prefetch past it is not used), one slot
  // ahead of the loads that need them.
  int row[8];
  auto find_rows = [&](int k) {
    const int p0 = lo + min(k, n - 1) * kSlotRows;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int p = p0 + 8 * lq + i < hi ? p0 + 8 * lq + i : p0;
      row[i] = plan.index ? plan.perm[p] : p;
    }
  };
  auto load = [&](int k, OuterSlot<NT, Q8>& o) {
    const int slot = first_slot + min(k, n - 1);
    o.e = exps[slot];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (Q8) {
        const uint2 c = *reinterpret_cast<const uint2*>(codes + static_cast<size_t>(row[i]) * C + cc);
        o.v[i] = uint4{c.x, c.y, 0, 0};
        const uint32_t sc = __builtin_bit_cast(uint16_t, xs[static_cast<size_t>(row[i]) * G + (cc >> gshift)]);
        if (i & 1) o.s2[i >> 1] |= sc << 16;
        else o.s2[i >> 1] = sc;
      } else {
        o.v[i] = *reinterpret_cast<const uint4*>(x + static_cast<size_t>(row[i]) * C + cc);
      }
    }
    const half8_t* f = reinterpret_cast<const half8_t*>(frags) + static_cast<size_t>(slot) * NTT * 128 + lane;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int tt = min(t0 + t, NTT - 1);   // past the last: computed, not stored
      o.h[t][0] = f[tt * 128];
      o.h[t][1] = f[tt * 128 + 64];
    }
  };

  float4_t acc[8][NT] = {};
  int E = kNoExponent;   // sums are in units of 2^E
  auto add = [&](OuterSlot<NT, Q8>& o) {
    const int e = __builtin_amdgcn_readfirstlane(o.e);
    if (e > E) {
      if (E != kNoExponent)
#pragma unroll
        for (int c = 0; c < 8; ++c)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[c][t][r] = __builtin_ldexpf(acc[c][t][r], E - e);
      E = e;
    } else if (e < E && e != kNoExponent) {
      const half_t down = static_cast<half_t>(__builtin_ldexpf(1.0f, max(e - E, -40)));
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        o.h[t][0] *= down;
        o.h[t][1] *= down;
      }
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      half8_t xf;
      if constexpr (Q8) {
        uint32_t d[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t e0 = c < 4 ? o.v[2 * i].x : o.v[2 * i].y, e1 = c < 4 ? o.v[2 * i + 1].x : o.v[2 * i + 1].y;
          // byte c % 4 of both rows into the low bytes of the two halves
          const uint32_t sel = 0x0C000C00u | static_cast<uint32_t>(c & 3) | (static_cast<uint32_t>(4 + (c & 3)) << 16);
          d[i] = act_value_pair(__builtin_amdgcn_perm(e1, e0, sel), as_h2(o.s2[i]));
        }
        xf = __builtin_bit_cast(half8_t, (u32x4_t{d[0], d[1], d[2], d[3]}));
      } else {
        xf = column8(o.v, c);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int p = 0; p < 2; ++p)
          acc[c][t] = CMAJOR ? __builtin_amdgcn_mfma_f32_16x16x32_f16(xf, o.h[t][p], acc[c][t], 0, 0, 0)
                             : __builtin_amdgcn_mfma_f32_16x16x32_f16(o.h[t][p], xf, acc[c][t], 0, 0, 0);
    }
  };

  if (n > 0) {
    OuterSlot<NT, Q8> ring[D];
    find_rows(wave);
#pragma unroll
    for (int d = 0; d < D; ++d) {
      load(wave + d * W, ring[d]);
      find_rows(wave + (d + 1) * W);
    }
    for (int k = wave; k < n; k += D * W) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (k + d * W >= n) break;
        add(ring[d]);
        load(k + (d + D) * W, ring[d]);
        find_rows(k + (d + D + 1) * W);
      }
    }
  }

  // Sum over the wavefronts, one channel fragment at a time, in units of 1.
  const float si = scaling ? scaling[ad] : 1.0f;
  float* g = grad + static_cast<size_t>(ad) * R * C;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float4_t v = acc[c][t];
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = __builtin_ldexpf(v[r], E);
      red[(wave * NT + t) * 64 + lane] = v;
    }
    __syncthreads();
    for (int i = tid; i < NT * 64; i += 64 * W) {
      float4_t v = red[i];
      for (int w = 1; w < W; ++w) v += red[w * NT * 64 + i];
      const int j0 = 16 * (t0 + i / 64);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int ch = CMAJOR ? c0 + 8 * (4 * ((i & 63) >> 4) + r) + c : c0 + 8 * (i & 15) + c;
        const int j = CMAJOR ? j0 + (i & 15) : j0 + 4 * ((i & 63) >> 4) + r;
        if (ch < C && j < R) g[CMAJOR ? static_cast<size_t>(ch) * R + j : static_cast<size_t>(j) * C + ch] = si * v[r];
      }
    }
  }
}

}  // namespace w4a16
