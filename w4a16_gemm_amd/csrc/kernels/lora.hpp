// Low-rank adapters of many requests beside a shared projection, and their gradients.
//
// Row m of the activations belongs to adapter i = index[m].  Forward:
//   h[m] = A_i x[m]                                  (shrink, K -> R)
//   out[m] = y[m] + s_i B_i h[m]                     (expand, R -> N)
// Backward:
//   g[m] = B_i^T dy[m]                               (shrink, N -> R)
//   dx[m] = dx0[m] + s_i A_i^T g[m]                  (expand, R -> K)
//   dB_i = s_i sum_m dy[m] h[m]^T,  dA_i = s_i sum_m g[m] x[m]^T       (outer)
//
// All of them are tall products with one side of R <= 128, on v_mfma_f32_16x16x32_f16
// with fp32 sums.  Every operand that comes from memory is binary16 and enters exactly.  (The
// instruction aligns the products it adds by their operands' exponents, a subnormal operand
// counting as 2^-14: measured, 2^-24 * 1 + 2^-24 * 2^-g comes out exact up to g = 14 and as 2^-24
// above.  Sums of products of subnormal values thus have steps of 2^-24 of what the products would
// be with operands of 2^-14.)  h and g are fp32 sums and enter as two binary16 terms (hi + lo)
// after a division by a power of two that brings the largest of them to [2^13, 2^14), so nothing
// overflows.  The two terms hold a value to 2^-23 of itself within 2^15 of that largest one: of a rank in a
// slot of 32 rows in the outer products, of a row in out and dx.  A slot or row with a smaller value
// that the terms do not hold is multiplied in fp32 (v_mfma_f32_16x16x4_f32).
//
// Rows are worked on in tiles of 16 to 128 rows of one adapter each; rows of one adapter are
// found through a row plan (below), so any order of rows costs the same products.
#pragma once

#include "act8.hpp"

namespace w4a16 {

// How rows are grouped by adapter.  Class of a row: its adapter, or L ("none") for an
// index outside [0, L).
//   index == NULL             every row belongs to adapter 0
//   off == NULL (M <= 256)    each workgroup groups the rows itself, one row per thread
//   else                      off[c] = first sorted position of class c (L + 2 entries),
//                             perm[p] = row at sorted position p (plan_rows_kernel)
struct RowPlan {
  const int32_t* index;
  const int32_t* off;
  const int32_t* perm;
  int M, L;
};

constexpr int kInlineRows = 256;

__device__ __forceinline__ int row_class(int i, int L) { return i >= 0 && i < L ? i : L; }

// Stable grouping by class: workgroup c counts the rows of smaller classes, then places
// its own rows in order.  No atomics, so the order (and with it every sum) is fixed.
// Latency-bound: 4 us for 2048 rows of eight adapters.  (Grouping inside the kernel that
// follows, beside workgroups that write the plan, cost that kernel as much.)
constexpr int kPlanRows = 8;   // rows per thread read at once (8192 per workgroup)

__global__ __launch_bounds__(1024) void plan_rows_kernel(const int32_t* __restrict__ index, int M, int L,
                                                         int32_t* __restrict__ off, int32_t* __restrict__ perm) {
  __shared__ int part[2][16];
  const int c = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int cls[kPlanRows];
  auto load = [&](int m0) {   // rows past M: a class above all
#pragma unroll
    for (int k = 0; k < kPlanRows; ++k) {
      const int m = m0 + 1024 * k + tid;
      cls[k] = m < M ? row_class(index[m], L) : L + 1;
    }
  };
  int below = 0;
  for (int m0 = 0; m0 < M; m0 += 1024 * kPlanRows) {
    load(m0);
#pragma unroll
    for (int k = 0; k < kPlanRows; ++k) below += cls[k] < c ? 1 : 0;
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) below += __shfl_xor(below, d);
  if (lane == 0) part[1][wave] = below;
  __syncthreads();
  int at = 0;
  for (int w = 0; w < 16; ++w) at += part[1][w];
  if (tid == 0) {
    off[c] = at;
    if (c == L) off[L + 1] = M;
  }
  __syncthreads();
  for (int m0 = 0; m0 < M; m0 += 1024 * kPlanRows) {
    if (M > 1024 * kPlanRows) load(m0);
#pragma unroll
    for (int k = 0; k < kPlanRows; ++k) {
      if (m0 + 1024 * k >= M) break;
      const bool mine = cls[k] == c;
      const uint64_t b = __ballot(mine);
      if (lane == 0) part[k & 1][wave] = __popcll(b);
      __syncthreads();   // the other half of part is free again once everyone is here
      int before = 0, total = 0;
      for (int w = 0; w < 16; ++w) {
        before += w < wave ? part[k & 1][w] : 0;
        total += part[k & 1][w];
      }
      if (mine) perm[at + before + __popcll(b & ((1ull << lane) - 1ull))] = m0 + 1024 * k + tid;
      at += total;
    }
  }
}

// Number of tile slots for T rows per tile.  With a plan in memory the slots of class c
// start at off[c] / T + c, which leaves room for every class's last partial tile.
__host__ __device__ inline int tile_slots(int M, int L, bool with_index, bool in_memory, int T) {
  if (!with_index) return (M + T - 1) / T;
  const int most = M / T + L + 1;
  return !in_memory && M < most ? M : most;
}

// Tiles found by one kernel for the next.
struct SlotTable {
  int2* meta;        // [slots] adapter (L: none), count (0: empty slot)
  int32_t* rows;     // [slots][rows per tile], entries past the count repeat a valid row
};

constexpr int kSlotRows = 32;    // of the split and stream kernels
constexpr int kFewRows = 16;     // of the kernels for few rows

struct Tile {
  int adapter;   // L: rows without an adapter
  int count;     // rows in the tile, 0: empty slot
};

// Tile of a slot; every thread of the workgroup (256 or more) calls it, `rows` (LDS, T
// entries) holds the tile's rows afterwards, entries past the count repeating a valid row.
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
    // The last class that starts at this slot or before; its starts increase with the class,
    // so 64 of them at a time narrow it down to a 64th (class 0 starts at slot 0).
    int c = 0;
    for (int step = p.L < 64 ? 1 : p.L < 4096 ? 64 : 4096;; step >>= 6) {
      const int k = c + lane * step;
      const int at = min(k, p.L);
      c += (__popcll(__ballot(k <= p.L && p.off[at] / T + at <= slot)) - 1) * step;
      if (step == 1) break;
    }
    const int lo = p.off[c], hi = p.off[c + 1];
    const int first = lo + (slot - (lo / T + c)) * T;
    t.adapter = c;
    t.count = max(0, min(T, hi - first));
    if (tid < T && t.count > 0) rows[tid] = p.perm[first + min(tid, t.count - 1)];
  } else if (p.M == 1) {
    t.adapter = row_class(p.index[0], p.L);
    t.count = slot == 0 ? 1 : 0;
    if (tid < T) rows[tid] = 0;
  } else {
    // Thread m counts the earlier rows of its class.  A tile starts at every T-th row of a
    // class; slots number the starts in the order of the rows.
    __shared__ __align__(16) int32_t cls[kInlineRows];
    __shared__ int32_t starts[4], start[2], members[4];
    const int wave = tid >> 6;
    if (tid < kInlineRows) cls[tid] = tid < p.M ? row_class(p.index[tid], p.L) : -1;
    if (tid < 2) start[tid] = 0;
    __syncthreads();
    const int mine = tid < p.M ? cls[tid] : -1;
    int rank = 0;
    for (int k0 = 0; k0 < p.M; k0 += 32) {
      int4 c[8];   // entries from M on are -1
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = *reinterpret_cast<const int4*>(cls + k0 + 4 * i);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = k0 + 4 * i;
        rank += (c[i].x == mine && k < tid) + (c[i].y == mine && k + 1 < tid) + (c[i].z == mine && k + 2 < tid) +
                (c[i].w == mine && k + 3 < tid);
      }
    }
    const bool starts_tile = mine >= 0 && rank % T == 0;
    const uint64_t sb = __ballot(starts_tile);
    if (lane == 0 && wave < 4) starts[wave] = __popcll(sb);
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < 4; ++w) {
      before += w < wave ? starts[w] : 0;
      total += starts[w];
    }
    if (starts_tile && before + __popcll(sb & ((1ull << lane) - 1ull)) == slot) {
      start[0] = tid;
      start[1] = rank;
    }
    __syncthreads();
    const int s = start[0], r0 = start[1];
    t.adapter = cls[s];
    const bool in = slot < total && mine == t.adapter && rank >= r0 && rank < r0 + T;
    const uint64_t mb = __ballot(in);
    if (lane == 0 && wave < 4) members[wave] = __popcll(mb);
    if (in) rows[rank - r0] = tid;
    __syncthreads();
    t.count = members[0] + members[1] + members[2] + members[3];
    if (tid < T && tid >= t.count) rows[tid] = s;
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

// v = h 2^shift as hi + lo in binary16.  An infinite or NaN h keeps it in hi alone.  Where lo
// is subnormal it holds multiples of 2^-24: a v of at least 2^-2 is still within 2^-23 of itself.
// Below, false is returned if anything is lost.  Sums of like products hardly ever lose: what is small
// beside the others is so by cancellation and has few bits (none of 128 slots of h or of g at rank 64).
__device__ __forceinline__ bool split_half(float h, int shift, half_t& hi, half_t& lo) {
  const float v = __builtin_ldexpf(h, shift);
  hi = static_cast<half_t>(v);
  const float r = v - static_cast<float>(hi);
  lo = static_cast<half_t>(__builtin_fabsf(v) <= 65504.0f ? r : 0.0f);
  return !(__builtin_fabsf(v) < 0.25f && static_cast<float>(lo) != r);
}

constexpr int kMaxRank = 128;
constexpr int kSplitTop = 14;   // split operands are below 2^14
constexpr int kLeastExponent = -148;   // of an outer operand: 2^e is an fp32 number, h 2^-e exact

// --- shrink: out[s][m][j] = sum over the channels of slice s of x[m][c] w[i][j][c] -------
//
// x [M][C], w [L][R][C], C % 8 == 0.  A wavefront holds 16 rows x 16 NT ranks of sums and
// walks steps of 32 channels, x as it lies in memory (lane (r, q): row r, channels 8 q ..
// 8 q + 7 of the step).  A row's result depends on its own x alone, so the rows repeated to
// fill a tile are computed and not stored.  Consecutive workgroups take the slices of one
// tile, so that an XCD's L2 holds the w of few slices.

// Steps [b, e) of 32 channels of 16 rows, dealt in pairs to W wavefronts, w as it lies in
// memory, D steps in flight.  xr: this lane's row; w [R][C].
template <int NT>
struct ShrinkStep {
  half8_t x, w[NT];
};

template <int NT, int W, int D>
__device__ __forceinline__ void shrink_steps(const half_t* __restrict__ xr, const half_t* __restrict__ w, int C, int R,
                                             int b, int e, int wave, int lane, float4_t (&acc)[NT]) {
  const int lr = lane & 15, lq = lane >> 4;
  const half_t* wr[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) wr[t] = w + static_cast<size_t>(min(16 * t + lr, R - 1)) * C;
  const int full = C >> 5;   // whole steps
  // Step k of this wavefront, of n.  Loads past the slice are clamped into it, not used.
  auto step_of = [&](int k) { return b + 2 * (wave + (k >> 1) * W) + (k & 1); };
  const int whole = (e - b) / (2 * W), rest = (e - b) % (2 * W);
  const int n = 2 * whole + max(0, min(2, rest - 2 * wave));
  auto load = [&](int k, ShrinkStep<NT>& o) {
    const int c = min(min(step_of(k), e - 1) * 32 + 8 * lq, C - 8);
    o.x = *reinterpret_cast<const half8_t*>(xr + c);
#pragma unroll
    for (int t = 0; t < NT; ++t) o.w[t] = *reinterpret_cast<const half8_t*>(wr[t] + c);
  };
  auto add = [&](int k, ShrinkStep<NT>& o) {
    const int st = step_of(k);
    if (st >= full) {   // the last, partial step: channels past C are zero on both sides
      const bool in = st * 32 + 8 * lq < C;
      o.x = in ? o.x : half8_t{};
#pragma unroll
      for (int t = 0; t < NT; ++t) o.w[t] = in ? o.w[t] : half8_t{};
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(o.x, o.w[t], acc[t], 0, 0, 0);
  };
  // The main loop reloads a stage as soon as it is used; the tail loads only what is left.
  ShrinkStep<NT> ring[D];
#pragma unroll
  for (int d = 0; d < D; ++d) load(d, ring[d]);
  int k = 0;
  for (; k + 2 * D <= n; k += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      add(k + d, ring[d]);
      load(k + d + D, ring[d]);
    }
  }
#pragma unroll
  for (int d = 0; d < D; ++d) {
    if (k + d < n) add(k + d, ring[d]);
    if (k + d + D < n) load(k + d + D, ring[d]);
  }
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (k + d + D < n) add(k + d + D, ring[d]);
}

// Sum of acc over the wavefronts of a workgroup, in a fixed order, left in wavefront 0.
// red: W / 2 * NT * 64 entries of LDS; every thread calls it.
template <int NT, int W>
__device__ __forceinline__ void add_wavefronts(float4_t* red, int wave, int lane, float4_t (&acc)[NT]) {
#pragma unroll
  for (int half = W / 2; half > 0; half >>= 1) {
    if (wave >= half && wave < 2 * half)
#pragma unroll
      for (int t = 0; t < NT; ++t) red[((wave - half) * NT + t) * 64 + lane] = acc[t];
    __syncthreads();
    if (wave < half)
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[t] += red[(wave * NT + t) * 64 + lane];
    __syncthreads();
  }
}

// Few rows: a tile of 16 rows and a slice per workgroup of 4 wavefronts.  table.meta != NULL:
// the next kernel works on the same tiles, so the tiles are written down and the sums go out
// by tile, [slots][S][16][R], where that kernel can read them without looking up rows.
// Latency-bound: 16 rows x 8192 of eight adapters at rank 16 5.4 us, 0.4 of them for the bytes.
template <int NT, int D>
__global__ __launch_bounds__(256) void lora_shrink_kernel(const half_t* __restrict__ x, const half_t* __restrict__ w,
                                                          RowPlan plan, int C, int R, int S, float* __restrict__ out,
                                                          SlotTable table) {
  constexpr int W = 4;
  __shared__ int32_t rows[kFewRows];
  __shared__ float4_t red[W / 2 * NT * 64];
  const int s = blockIdx.x % S, slot = blockIdx.x / S;
  const bool by_slot = table.meta != nullptr;
  const Tile tile = find_tile<kFewRows>(plan, slot, rows);
  const int tid = threadIdx.x, lane = tid & 63;
  if (by_slot && s == 0) {
    if (tid == 0) table.meta[slot] = int2{tile.adapter, tile.count};
    if (tid < kFewRows && tile.count > 0) table.rows[slot * kFewRows + tid] = rows[tid];
  }
  if (tile.count == 0 || (by_slot && tile.adapter == plan.L)) return;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lq = lane >> 4;
  float* o = out + static_cast<size_t>(s) * plan.M * R;
  if (tile.adapter == plan.L) {
    for (int i = tid; i < tile.count * R; i += 64 * W) o[static_cast<size_t>(rows[i / R]) * R + i % R] = 0.0f;
    return;
  }
  const int steps = (C + 31) >> 5;
  const int b = static_cast<int>(static_cast<int64_t>(steps) * s / S);
  const int e = static_cast<int>(static_cast<int64_t>(steps) * (s + 1) / S);
  float4_t acc[NT] = {};
  shrink_steps<NT, W, D>(x + static_cast<size_t>(rows[lr]) * C, w + static_cast<size_t>(tile.adapter) * R * C, C, R, b, e,
                         wave, lane, acc);
  add_wavefronts<NT, W>(red, wave, lane, acc);
  if (wave != 0) return;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = 4 * lq + r, j = 16 * t + lr;
      float* to = by_slot ? out + (static_cast<size_t>(blockIdx.x) * kFewRows + i) * R : o + static_cast<size_t>(rows[i]) * R;
      if (i < tile.count && j < R) to[j] = acc[t][r];
    }
}

// Many rows: HBM-bound on x.  A tile of 16 W rows per workgroup, 16 per wavefront, so that w
// is read once per tile; it goes through LDS (two buffers of 64 channels in operand order,
// 16-byte accesses) while x and w stream into registers D chunks ahead: 4096 rows x 28672
// channels at rank 64 in 51 us, 4.6 TB/s (with D = 2 54 us; eight operands of 16 ranks leave
// registers for no more).  With w read by every wavefront for itself the
// kernel was bound by L2 traffic: 83 us with 64 rows per wavefront, 138 us with 16.
// The barrier orders LDS only: the x and w loads in flight pass it.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// TRANS: w is [L][C][R] (the b of the forward): it comes from memory as 8 ranks of a channel,
// and takes its operand order on the way into LDS (16-bit writes, 8 per 16 bytes; the
// operands' padding keeps the 16 pieces of a channel on different banks).
template <int NT, int W, bool TRANS, int D>
__global__ __launch_bounds__(64 * W) void lora_shrink_tall_kernel(const half_t* __restrict__ x,
                                                                  const half_t* __restrict__ w, RowPlan plan, int C,
                                                                  int R, int S, float* __restrict__ out) {
  constexpr int T = 16 * W, SC = 2;                       // steps per chunk
  constexpr int kPieces = NT * 16 * SC * 4;               // 16-byte pieces of w per chunk
  constexpr int PT = (kPieces + 64 * W - 1) / (64 * W);   // per thread
  __shared__ int32_t rows[T];
  constexpr int TS = 65;                                  // operand of a step and 16 ranks, padded
  __shared__ half8_t lds[2][SC * NT * TS];
  const int s = blockIdx.x % S;
  const Tile tile = find_tile<T>(plan, blockIdx.x / S, rows);
  if (tile.count == 0) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lq = lane >> 4;
  float* o = out + static_cast<size_t>(s) * plan.M * R;
  if (tile.adapter == plan.L) {
    for (int i = tid; i < tile.count * R; i += 64 * W) o[static_cast<size_t>(rows[i / R]) * R + i % R] = 0.0f;
    return;
  }
  const half_t* xr = x + static_cast<size_t>(rows[16 * wave + lr]) * C;
  const half_t* wl = w + static_cast<size_t>(tile.adapter) * R * C;
  const int chunks = (C + 32 * SC - 1) / (32 * SC);
  const int b = static_cast<int>(static_cast<int64_t>(chunks) * s / S);
  const int e = static_cast<int>(static_cast<int64_t>(chunks) * (s + 1) / S);
  float4_t acc[NT] = {};
  half8_t wreg[D][PT];
  half8_t xs[D][SC];
  // Pieces of 8 values of w per thread: ranks or channels of the chunk, and which.
  const int octs = TRANS ? R >> 3 : SC * 4;   // pieces per channel or rank
  int line[PT], oct[PT];
#pragma unroll
  for (int i = 0; i < PT; ++i) {
    line[i] = (tid + 64 * W * i) / octs;
    oct[i] = (tid + 64 * W * i) % octs;
  }
  // Loads past the slice or past C are clamped; channels past C are zeroed on both sides.
  auto load_w = [&](int k, half8_t (&v)[PT]) {
    const int cb = min(k, e - 1) * 32 * SC;
#pragma unroll
    for (int i = 0; i < PT; ++i) {
      const size_t at = TRANS ? static_cast<size_t>(min(cb + line[i], C - 1)) * R + 8 * oct[i]
                              : static_cast<size_t>(min(line[i], R - 1)) * C + min(cb + 8 * oct[i], C - 8);
      v[i] = *reinterpret_cast<const half8_t*>(wl + at);
    }
  };
  auto store_w = [&](int k, int buf, const half8_t (&w8)[PT]) {
#pragma unroll
    for (int i = 0; i < PT; ++i) {
      if constexpr (TRANS) {
        const int c = line[i];   // channel of the chunk
        if (c >= 32 * SC) continue;
        const half8_t v = k * 32 * SC + c < C ? w8[i] : half8_t{};
        half_t* to = reinterpret_cast<half_t*>(lds[buf]) + (((c >> 5) * NT * TS + ((c >> 3) & 3) * 16) * 8 + (c & 7));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int rank = 8 * oct[i] + j;
          to[((rank >> 4) * TS + (rank & 15)) * 8] = v[j];
        }
      } else {
        const int j = line[i], q = oct[i];
        if (j >= 16 * NT) continue;
        lds[buf][((q >> 2) * NT + (j >> 4)) * TS + (q & 3) * 16 + (j & 15)] =
            k * 32 * SC + 8 * q < C ? w8[i] : half8_t{};
      }
    }
  };
  auto load_x = [&](int k, half8_t (&v)[SC]) {
#pragma unroll
    for (int u = 0; u < SC; ++u)
      v[u] = *reinterpret_cast<const half8_t*>(xr + min(min(k, e - 1) * 32 * SC + 32 * u + 8 * lq, C - 8));
  };
  auto add = [&](int k, int buf, half8_t (&v)[SC]) {
    if ((k + 1) * 32 * SC > C)
#pragma unroll
      for (int u = 0; u < SC; ++u) v[u] = k * 32 * SC + 32 * u + 8 * lq < C ? v[u] : half8_t{};
#pragma unroll
    for (int u = 0; u < SC; ++u)
#pragma unroll
      for (int t = 0; t < NT; ++t)
        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v[u], lds[buf][(u * NT + t) * TS + lane], acc[t], 0, 0, 0);
  };
  // Chunk k: x in xs[k % D] (from b on), w in wreg[k % D] until it is in LDS.  Loads complete
  // in order, so w is as far ahead as x.
#pragma unroll
  for (int d = 0; d < D; ++d) {
    load_w(b + d, wreg[d]);
    load_x(b + d, xs[d]);
  }
  store_w(b, 0, wreg[0]);
  load_w(b + D, wreg[0]);
  lds_barrier();
  auto step = [&](int k, int d, bool inside) {   // d = (k - b) % D; inside: nothing ends yet
    add(k, d & 1, xs[d]);
    if (inside || k + D < e) load_x(k + D, xs[d]);
    if (inside || k + 1 < e) store_w(k + 1, (d + 1) & 1, wreg[(d + 1) % D]);
    if (inside || k + 1 + D < e) load_w(k + 1 + D, wreg[(d + 1) % D]);
    lds_barrier();
  };
  int k = b;
  for (; k + 2 * D < e; k += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) step(k + d, d, true);
  }
#pragma unroll
  for (int d = 0; d < 2 * D; ++d)
    if (k + d < e) step(k + d, d % D, false);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = 16 * wave + 4 * lq + r, j = 16 * t + lr;
      if (i < tile.count && j < R) o[static_cast<size_t>(rows[i]) * R + j] = acc[t][r];
    }
}

// --- expand: out[m][c] = binary16(base[m][c] + s_i sum_j h[m][j] w_i[c][j]) ---------------
//
// One operand of an MFMA is 16 rows x 32 ranks of h, the other 32 ranks x 16 channels of the
// weights; a wavefront holds the weights of 128 channels (8 tiles).  Two arrangements:
//   many rows   h is the A operand; column r of tile t is channel 8 r + t, so a lane (r, q)
//               ends up with 8 consecutive channels of each of the rows 4 q .. 4 q + 3, and
//               base and out move as 16-byte accesses of 256 consecutive bytes per row.
//               w [L][C][R], or TRANS: w [L][R][C], where lane (r, q) loads octet r of its 8
//               ranks and transposes the 8 x 8 block in registers.
//   few rows    the weights are the A operand; row 4 q + r of tile t is channel 32 (t / 2) +
//               8 q + 4 (t % 2) + r, so a lane has four runs of 8 channels (at 32 u + 8 q) of
//               row r: 64 bytes of a row per access, but the weights, here the larger part,
//               are read as 4 whole rows of w (the first arrangement reads every eighth).
// Measured: 4096 rows x 28672 channels at rank 64 94 us in the first, 114 us in the second;
// one row, 1536 channels, rank 16 (whole forward) 7.2 us in the first, 6.0 us in the second.
// R <= 16 (PACKED): hi and lo share one MFMA, ranks 0..15 of hi in its first 16 slots and
// of lo in the last 16, against the same weights.  Larger R: F fragments of 32 ranks,
// one MFMA for hi and one for lo each.

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

// Sum of S slices of ROWS x R floats into LDS: sums[m (R / 4 + 1) + j] holds ranks 4 j .. of
// row m, zero from row `count` on.  at(m): offset of row m in a slice.  Where R leaves threads
// over, groups of them take every G-th slice each, and their sums are added in order.  Every
// thread calls it; `sums` has room for sum_quads(ROWS, THREADS) entries.
constexpr int sum_quads(int rows, int threads) {
  // rows (kMaxRank / 4 + 1) for one group; G rows (R / 4 + 1) with G = threads / (rows R / 4)
  const int one = rows * (kMaxRank / 4 + 1), most = threads + threads / 2;   // R >= 8: (R / 4 + 1) / (R / 4) <= 3 / 2
  return one > most ? one : most;
}

template <int ROWS, int THREADS, typename At>
__device__ __forceinline__ void sum_slices(const float* __restrict__ h, size_t slice, int S, int R, int count,
                                           float4_t* sums, At at) {
  const int tid = threadIdx.x;
  const int quads = R >> 2, ld = quads + 1, items = ROWS * quads;
  const int G = min(max(1, THREADS / items), S);
  constexpr int U = 8;   // slices in flight
  for (int i = tid; i < items * G; i += THREADS) {
    const int g = i / items, m = i % items / quads, j = i % quads;
    float4_t v = {};
    if (m < count) {
      const float* p = h + at(m) + 4 * j;
      for (int s0 = g; s0 < S; s0 += U * G) {
        float4_t q[U];
#pragma unroll
        for (int k = 0; k < U; ++k) q[k] = *reinterpret_cast<const float4_t*>(p + min(s0 + k * G, S - 1) * slice);
#pragma unroll
        for (int k = 0; k < U; ++k)
          if (s0 + k * G < S) v += q[k];
      }
    }
    sums[(g * ROWS + m) * ld + j] = v;
  }
  __syncthreads();
  if (G == 1) return;
  for (int i = tid; i < items; i += THREADS) {
    const int at0 = i / quads * ld + i % quads;
    float4_t v = sums[at0];
    for (int g = 1; g < G; ++g) v += sums[g * ROWS * ld + at0];
    sums[at0] = v;
  }
  __syncthreads();
}

// Weights of the 128 channels from c0 (channels past C repeat valid ones), in the order of
// many rows or of few.
template <int F, bool PACKED, bool TRANS, bool MANY>
__device__ __forceinline__ void load_expand_weights(const half_t* __restrict__ w, int c0, int C, int R, int lane,
                                                    half8_t (&wf)[F][8]) {
  static_assert(MANY || !TRANS, "few rows read w [L][C][R]");
  const int lr = lane & 15, lq = lane >> 4;
#pragma unroll
  for (int f = 0; f < F; ++f) {
    const int j0 = PACKED ? (lq & 1) * 8 : 32 * f + 8 * lq;
    const bool in = j0 < R;
    if constexpr (!TRANS) {
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const int c = min(c0 + (MANY ? 8 * lr + t : 32 * (t >> 1) + 8 * (lr >> 2) + 4 * (t & 1) + (lr & 3)), C - 1);
        const half8_t v = *reinterpret_cast<const half8_t*>(w + static_cast<size_t>(c) * R + (in ? j0 : 0));
        wf[f][t] = in ? v : half8_t{};
      }
    } else {
      const int cc = min(c0 + 8 * lr, C - 8);
      uint4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = *reinterpret_cast<const uint4*>(w + static_cast<size_t>(in ? j0 + i : i) * C + cc);
        if (!in) v[i] = uint4{0, 0, 0, 0};
      }
#pragma unroll
      for (int t = 0; t < 8; ++t) wf[f][t] = column8(v, t);
    }
  }
}

// Products of one group of 16 rows with the weights, in fp32 (8 times the cycles): v holds this
// lane's ranks of row r, in the order of its operands.
template <int F, bool PACKED, bool MANY>
__device__ __forceinline__ void expand_products_fp32(const half8_t (&wf)[F][8], const float (&v)[F][8], int lq,
                                                     float4_t (&acc)[8]) {
#pragma unroll
  for (int t = 0; t < 8; ++t) acc[t] = float4_t{};
#pragma unroll
  for (int f = 0; f < F; ++f)
#pragma unroll
    for (int i = 0; i < 8; ++i) {   // step i: ranks 8 q + i of every quarter q
      const float h = PACKED && lq >= 2 ? 0.0f : v[f][i];
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const float w = PACKED && lq >= 2 ? 0.0f : static_cast<float>(wf[f][t][i]);
        acc[t] = MANY ? __builtin_amdgcn_mfma_f32_16x16x4f32(h, w, acc[t], 0, 0, 0)
                      : __builtin_amdgcn_mfma_f32_16x16x4f32(w, h, acc[t], 0, 0, 0);
      }
      __builtin_amdgcn_sched_barrier(0);   // one step's weights in registers at a time
    }
}

// Products of one fragment of 16 rows with the weights, added to acc.
template <int P, bool MANY>
__device__ __forceinline__ void expand_products(const half8_t (&wf)[8], const half8_t (&hf)[P], float4_t (&acc)[8]) {
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int t = 0; t < 8; ++t)
      acc[t] = MANY ? __builtin_amdgcn_mfma_f32_16x16x32_f16(hf[p], wf[t], acc[t], 0, 0, 0)
                    : __builtin_amdgcn_mfma_f32_16x16x32_f16(wf[t], hf[p], acc[t], 0, 0, 0);
}

// 8 consecutive results of a lane: row 4 q + u (many rows), run u (few rows).
template <bool MANY>
__device__ __forceinline__ half8_t expand_result(const float4_t (&acc)[8], int u, uint4 y, float factor) {
  const half8_t yv = __builtin_bit_cast(half8_t, y);
  half8_t o;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    o[i] = static_cast<half_t>(fmaf(MANY ? acc[i][u] : acc[2 * u + (i >> 2)][i & 3], factor, static_cast<float>(yv[i])));
  return o;
}

// This lane's ranks of its row.
template <int F, bool PACKED>
__device__ __forceinline__ void load_ranks(const float* row, int R, int lq, float (&v)[F][8]) {
#pragma unroll
  for (int f = 0; f < F; ++f) {
    const int j0 = PACKED ? (lq & 1) * 8 : 32 * f + 8 * lq;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[f][j] = j0 < R ? row[j0 + j] : 0.0f;
  }
}

// Of a ballot over lanes (r, q), the 16 rows r.
__device__ __forceinline__ uint32_t wide_rows(uint64_t lanes) {
  lanes |= lanes >> 32;
  return static_cast<uint32_t>(lanes | lanes >> 16) & 0xFFFFu;
}

// Few rows: 16 of them (row: that of lane (r, q), in LDS) with the weights.  Returns the factor
// that acc is still to be multiplied with.
template <int F, bool PACKED>
__device__ __forceinline__ float split_and_expand(const half8_t (&wf)[F][8], const float* row, int R, int lq, float si,
                                                  float4_t (&acc)[8]) {
  float v[F][8];
  load_ranks<F, PACKED>(row, R, lq, v);
  float top = 0.0f;
#pragma unroll
  for (int f = 0; f < F; ++f)
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, finite_magnitude(v[f][j]));
  top = fmaxf(top, __shfl_xor(top, 16));
  top = fmaxf(top, __shfl_xor(top, 32));
  const int shift = kSplitTop - top_exponent(top);
  bool whole = true;
#pragma unroll
  for (int t = 0; t < 8; ++t) acc[t] = float4_t{};
#pragma unroll
  for (int f = 0; f < F; ++f) {
    half8_t hf[PACKED ? 1 : 2];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      half_t hi, lo;
      whole &= split_half(v[f][j], shift, hi, lo);
      hf[0][j] = PACKED && lq >= 2 ? lo : hi;
      if constexpr (!PACKED) hf[1][j] = lo;
    }
    expand_products<PACKED ? 1 : 2, false>(wf[f], hf, acc);
  }
  const float factor = __builtin_ldexpf(si, -shift);
  const uint64_t wide = __ballot(!whole);
  if (!wide) return factor;
  asm volatile("" ::: "memory");   // read again here, not held in registers meanwhile
  load_ranks<F, PACKED>(row, R, lq, v);
  float4_t fp32[8];
  expand_products_fp32<F, PACKED, false>(wf, v, lq, fp32);
  const bool mine = wide_rows(wide) >> (threadIdx.x & 15) & 1;   // the others do not depend on them
#pragma unroll
  for (int t = 0; t < 8; ++t) acc[t] = mine ? fp32[t] : acc[t];
  return mine ? si : factor;
}

// --- split: h or g (the sum of S slices) as ready MFMA operands ---------------------------
//
// Latency-bound (5 - 8 us; 4096 rows at rank 64, eight slices, all loaded at once: 6.4 us).
// One workgroup per slot of 32 rows of one adapter and task, once per call instead of by
// every workgroup of 128 channels that multiplies with h.  The sum goes through LDS, from
// where it is written in either or both of two orders:
//   by_rank (outer)   fragment t: lane (r, q) has rank 16 t + r of rows 8 q .. 8 q + 7, in
//                     units of |unit| of that slot and rank, a power of two (ranks never meet in
//                     a gradient); [slots][NT][hi, lo][64][8].  A fragment that holds a value
//                     which two terms beside the largest of its rank cannot hold has negative units
//   by_row (stream)   group g of 16 rows, fragment f: lane (r, q) has ranks 32 f + 8 q .. + 7
//                     of row 16 g + r, in units of 2^e of that row, with factors[row of the
//                     slot] = s_i 2^e; [slots][2][F][hi, lo][64][8].  R <= 16: one fragment
//                     with hi of ranks 0 .. 15 in its first two quarters and lo in the
//                     others; [slots][2][64][8].  Bit r of wide[slot][f][g]: row 16 g + r has a
//                     value that two terms beside its largest one cannot hold
// Rows past the slot's count and ranks past R are zero.  A by-row task also writes the slot
// table.  Where wanted, the summed h is written (0 for rows without an adapter).
struct SplitTask {
  const float* h;    // [S][M][R]
  int S;
  half_t* by_rank;   // or NULL
  float* units;      // [slots][16 NT]
  half_t* by_row;    // or NULL
  float* factors;    // [slots][32]
  uint16_t* wide;    // [slots][4][2]
  float* sum;        // [M][R]: the summed h, or NULL
  float* far;        // [M][R]: the same of the slots that are not whole, or NULL
};

// By-row operands (of 1 KB) of a row group.
__host__ __device__ constexpr int row_frags(int R) { return R <= 16 ? 1 : 2 * ((R + 31) / 32); }

__global__ __launch_bounds__(512) void lora_split_kernel(SplitTask t0, SplitTask t1, const float* __restrict__ scaling,
                                                         SlotTable table, RowPlan plan, int R) {
  __shared__ int32_t rows[kSlotRows];
  __shared__ float row_top[kSlotRows];
  __shared__ float4_t sums[sum_quads(kSlotRows, 512)];
  const SplitTask task = blockIdx.y == 0 ? t0 : t1;
  const int slot = blockIdx.x;
  const Tile tile = find_tile<kSlotRows>(plan, slot, rows);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lr = lane & 15, lq = lane >> 4;
  const size_t slice = static_cast<size_t>(plan.M) * R;
  if (task.by_row) {
    if (tid == 0) table.meta[slot] = int2{tile.adapter, tile.count};
    if (tid < kSlotRows && tile.count > 0) table.rows[slot * kSlotRows + tid] = rows[tid < tile.count ? tid : 0];
  }
  if (tile.count == 0) return;
  if (tile.adapter == plan.L) {
    if (task.sum)
      for (int i = tid; i < tile.count * R; i += 512) task.sum[static_cast<size_t>(rows[i / R]) * R + i % R] = 0.0f;
    return;
  }
  const int quads = R >> 2, ld = quads + 1;
  sum_slices<kSlotRows, 512>(task.h, slice, task.S, R, tile.count, sums,
                             [&](int m) { return static_cast<size_t>(rows[m]) * R; });
  if (task.sum)
    for (int i = tid; i < tile.count * quads; i += 512)
      *reinterpret_cast<float4_t*>(task.sum + static_cast<size_t>(rows[i / quads]) * R + 4 * (i % quads)) =
          sums[i / quads * ld + i % quads];
  const float* f = reinterpret_cast<const float*>(sums);
  auto keep = [&] {   // by the wavefront that finds a value, for those that multiply in fp32
    if (task.far)
      for (int i = lane; i < tile.count * quads; i += 64)
        *reinterpret_cast<float4_t*>(task.far + static_cast<size_t>(rows[i / quads]) * R + 4 * (i % quads)) =
            sums[i / quads * ld + i % quads];
  };
  if (task.by_rank) {
    const int NT = (R + 15) >> 4;
    for (int t = wave; t < NT; t += 8) {
      const int j = 16 * t + lr;
      float v[8], top = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = j < R ? f[(8 * lq + i) * 4 * ld + j] : 0.0f;
        top = fmaxf(top, finite_magnitude(v[i]));
      }
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const int e = top > 0.0f ? max(top_exponent(top) - kSplitTop, kLeastExponent) : 0;
      bool whole = true;
      half8_t hi, lo;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        half_t a, b;
        whole &= split_half(v[i], -e, a, b);
        hi[i] = a;
        lo[i] = b;
      }
      half8_t* o = reinterpret_cast<half8_t*>(task.by_rank) + (static_cast<size_t>(slot) * NT + t) * 128 + lane;
      o[0] = hi;
      o[64] = lo;
      const float unit = __builtin_ldexpf(1.0f, e);
      const bool all = __all(whole);
      if (lq == 0) task.units[(static_cast<size_t>(slot) * NT + t) * 16 + lr] = all ? unit : -unit;
      if (!all) keep();
    }
  }
  if (!task.by_row) return;
  // largest of every row: 16 threads per row
  {
    const int m = tid >> 4;
    float rt = 0.0f;
    for (int j = tid & 15; j < R; j += 16) rt = fmaxf(rt, finite_magnitude(f[m * 4 * ld + j]));
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) rt = fmaxf(rt, __shfl_xor(rt, d));
    if ((tid & 15) == 0) {
      row_top[m] = rt;
      const float si = scaling ? scaling[tile.adapter] : 1.0f;
      task.factors[slot * kSlotRows + m] = __builtin_ldexpf(si, top_exponent(rt) - kSplitTop);
    }
  }
  __syncthreads();
  const bool packed = R <= 16;
  const int F = packed ? 1 : (R + 31) / 32;
  for (int i = wave; i < 2 * F; i += 8) {   // operand pairs (row group, fragment)
    const int g = i / F, k = i % F;
    const int m = 16 * g + lr;
    const int j0 = packed ? 8 * (lq & 1) : 32 * k + 8 * lq;
    const int shift = kSplitTop - top_exponent(row_top[m]);
    bool whole = true;
    half8_t hi, lo;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      half_t a, b;
      whole &= split_half(j0 < R ? f[m * 4 * ld + j0 + j] : 0.0f, shift, a, b);
      hi[j] = packed && lq >= 2 ? b : a;
      lo[j] = b;
    }
    half8_t* o = reinterpret_cast<half8_t*>(task.by_row) + ((static_cast<size_t>(slot) * 2 + g) * row_frags(R)) * 64 + lane;
    if (packed) {
      o[0] = hi;
    } else {
      o[2 * k * 64] = hi;
      o[(2 * k + 1) * 64] = lo;
    }
    const uint32_t wide = wide_rows(__ballot(!whole));
    if (lane == 0) task.wide[slot * 8 + k * 2 + g] = static_cast<uint16_t>(wide);
    if (wide) keep();
  }
}

// --- expand, few rows: sums and splits h itself -------------------------------------------
//
// h by tile, [slots][S][16][R], and the tiles as the shrink wrote them.  A workgroup of 4
// wavefronts takes one tile of 16 rows x 512 channels; h is summed into LDS by all of it
// while the weights and base are on their way, and every wavefront splits it for itself.
// Latency-bound: what counts is one launch less, and few loads that wait for another (16 rows
// x 28672 of eight adapters at rank 16: 6.8 us).  Two workgroups per compute unit up to rank 32 (256
// rows x 11008 of 16 adapters at rank 16, whole forward: 18.4 us, without the bound 20.4 us); above, the
// registers go to the loads (64 rows of 8 adapters at rank 128: 21.6 us, with the bound 25.4 us; 16
// rows x 28672 at rank 64: 18.1 us, with it 19.8 us).
// base may equal out (every element is read and written by the same lane); rows without
// an adapter are copied, bit for bit.  h_out (not NULL): the workgroups of the first
// channels write the summed h.
template <int F, bool PACKED>
__global__ __launch_bounds__(256, F == 1 ? 2 : 1) void lora_expand_kernel(
    const float* __restrict__ h, int S, SlotTable table, const half_t* __restrict__ w, const float* __restrict__ scaling,
    int L, const half_t* base, half_t* out, float* __restrict__ h_out, int C, int R) {
  constexpr int kBlock = 512;   // channels per workgroup: 4 wavefronts x 128
  __shared__ float4_t sums[sum_quads(kFewRows, 256)];
  const int slot = blockIdx.x;
  const int2 meta = table.meta[slot];
  const int adapter = __builtin_amdgcn_readfirstlane(meta.x), count = __builtin_amdgcn_readfirstlane(meta.y);
  if (count == 0) return;
  const int32_t* rows = table.rows + slot * kFewRows;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lq = lane >> 4;
  const int c_lo = blockIdx.y * kBlock;
  if (adapter == L) {
    if (base != out) {
      const int chunks = min(kBlock, C - c_lo) / 8;
      for (int i = tid; i < count * chunks; i += 256) {
        const size_t at = static_cast<size_t>(rows[i / chunks]) * C + c_lo + 8 * (i % chunks);
        *reinterpret_cast<uint4*>(out + at) = *reinterpret_cast<const uint4*>(base + at);
      }
    }
    if (h_out && blockIdx.y == 0)
      for (int i = tid; i < count * R; i += 256) h_out[static_cast<size_t>(rows[i / R]) * R + i % R] = 0.0f;
    return;
  }
  const int c0 = c_lo + wave * 128;
  const size_t at = static_cast<size_t>(rows[lr]);
  uint4 y[4];
  half8_t wf[F][8];
  if (c0 < C) {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      y[u] = *reinterpret_cast<const uint4*>(base + at * C + min(c0 + 32 * u + 8 * lq, C - 8));
    load_expand_weights<F, PACKED, false, false>(w + static_cast<size_t>(adapter) * R * C, c0, C, R, lane, wf);
  }
  const int quads = R >> 2, ld = quads + 1;
  sum_slices<kFewRows, 256>(h + static_cast<size_t>(slot) * S * kFewRows * R, static_cast<size_t>(kFewRows) * R, S, R, count,
                            sums, [&](int m) { return static_cast<size_t>(m) * R; });
  if (h_out && blockIdx.y == 0)
    for (int i = tid; i < count * quads; i += 256)
      *reinterpret_cast<float4_t*>(h_out + static_cast<size_t>(rows[i / quads]) * R + 4 * (i % quads)) =
          sums[i / quads * ld + i % quads];
  if (c0 >= C) return;
  const float* hs = reinterpret_cast<const float*>(sums) + lr * 4 * ld;
  float4_t acc[8];
  const float factor = split_and_expand<F, PACKED>(wf, hs, R, lq, scaling ? scaling[adapter] : 1.0f, acc);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int c = c0 + 32 * u + 8 * lq;
    const half8_t o = expand_result<false>(acc, u, y[u], factor);
    if (c < C && lr < count) *reinterpret_cast<half8_t*>(out + at * C + c) = o;
  }
}

// --- forward of few rows in one launch ----------------------------------------------------
//
// Every workgroup (8 wavefronts, one tile of 16 rows x 1024 channels) computes h of its
// tile for itself: R K weights more from the L2 per workgroup, against a launch and a round
// trip of h through memory.  Weights and base of the wavefront's 128 channels are requested
// first and arrive during the shrink.
template <int F, bool PACKED, int D>
__global__ __launch_bounds__(512) void lora_fused_kernel(const half_t* __restrict__ x, const half_t* __restrict__ a,
                                                         const half_t* __restrict__ w,
                                                         const float* __restrict__ scaling, RowPlan plan,
                                                         const half_t* base, half_t* out, float* __restrict__ h_out,
                                                         int K, int N, int R) {
  constexpr int W = 8, NT = PACKED ? 1 : 2 * F;
  constexpr int ld = 16 * NT + 4;   // floats per row of h
  __shared__ int32_t rows[kFewRows];
  __shared__ float4_t red[W / 2 * NT * 64];
  __shared__ __align__(16) float hs[16 * ld];
  const int blocks = (N + 128 * W - 1) / (128 * W);
  const Tile tile = find_tile<kFewRows>(plan, blockIdx.x / blocks, rows);
  if (tile.count == 0) return;
  const int block = blockIdx.x % blocks;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lq = lane >> 4;
  if (tile.adapter == plan.L) {
    const int c_lo = block * 128 * W;
    if (base != out) {
      const int chunks = min(128 * W, N - c_lo) / 8;
      for (int i = tid; i < tile.count * chunks; i += 64 * W) {
        const size_t at = static_cast<size_t>(rows[i / chunks]) * N + c_lo + 8 * (i % chunks);
        *reinterpret_cast<uint4*>(out + at) = *reinterpret_cast<const uint4*>(base + at);
      }
    }
    if (h_out && block == 0)
      for (int i = tid; i < tile.count * R; i += 64 * W) h_out[static_cast<size_t>(rows[i / R]) * R + i % R] = 0.0f;
    return;
  }
  const int c0 = (block * W + wave) * 128;
  const size_t at = static_cast<size_t>(rows[lr]);
  uint4 y[4];
  half8_t wf[F][8];
  if (c0 < N) {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      y[u] = *reinterpret_cast<const uint4*>(base + at * N + min(c0 + 32 * u + 8 * lq, N - 8));
    load_expand_weights<F, PACKED, false, false>(w + static_cast<size_t>(tile.adapter) * R * N, c0, N, R, lane, wf);
  }

  float4_t acc[NT] = {};
  shrink_steps<NT, W, D>(x + at * K, a + static_cast<size_t>(tile.adapter) * R * K, K, R, 0, (K + 31) >> 5, wave, lane, acc);
  add_wavefronts<NT, W>(red, wave, lane, acc);
  if (wave == 0)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) hs[(4 * lq + r) * ld + 16 * t + lr] = acc[t][r];
  __syncthreads();
  if (h_out && block == 0)
    for (int i = tid; i < tile.count * R; i += 64 * W)
      h_out[static_cast<size_t>(rows[i / R]) * R + i % R] = hs[(i / R) * ld + i % R];
  if (c0 >= N) return;
  float4_t sums[8];
  const float factor = split_and_expand<F, PACKED>(wf, hs + lr * ld, R, lq, scaling ? scaling[tile.adapter] : 1.0f, sums);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int c = c0 + 32 * u + 8 * lq;
    const half8_t o = expand_result<false>(sums, u, y[u], factor);
    if (c < N && lr < tile.count) *reinterpret_cast<half8_t*>(out + at * N + c) = o;
  }
}

// --- expand, many rows: a stream over slots of 32 rows ------------------------------------
//
// HBM-bound: 2 bytes read and 2 written per element.  Operands come ready from the split
// kernel, so the wavefronts share nothing: no LDS, no barrier.  A wavefront takes `group`
// (at most 64) consecutive slots; slots of one adapter are a run with the weights in
// registers and the operands and base values of the next D row groups in flight.  The
// workgroups of one group of slots are neighbours, so an XCD's L2 holds few channels of w.
// base may equal out, or be absent (BASE == false: 0); rows without an adapter are copied.
// Rows that the split marked as wide are multiplied in fp32 after all the others, from the summed h
// (in groups of 16, but stored alone: a row's result depends on its own values).  Where there are none, looking for them costs 29.1 -> 29.5 us for 2048 rows x 14336 of
// eight adapters at rank 64 (31.5 us with their products at the end of each run), 94.0 -> 94.7 us
// for 4096 x 28672.
// out is written past the L2 (nobody reads it here): with plain stores 4096 x 28672 took 99 us
// against 94 us; 2048 rows x 14336 at rank 16 25.3 us against 19.6 us.
template <int F, int P>
struct StreamRows {
  uint4 y[4];
  half8_t h[F][P];
  int4 row;          // rows 4 q .. 4 q + 3 of the group
  float4_t factor;
};

__device__ __forceinline__ void store_past_l2(half_t* p, half8_t v) {
  __builtin_nontemporal_store(__builtin_bit_cast(u32x4_t, v), reinterpret_cast<u32x4_t*>(p));
}

struct StreamArgs {
  const half_t* frags;
  const float* factors;
  const uint16_t* wide;
  const float* h;          // [M][R], summed
  const float* scaling;
  SlotTable table;
  const half_t* w;
  const half_t* base;
  half_t* out;
  int C, R, L, slots, group;
};

template <int F, bool PACKED, bool TRANS, bool BASE, int D>
__device__ __forceinline__ void stream_rows(const StreamArgs& args, int block) {
  constexpr int P = PACKED ? 1 : 2;
  const half_t* __restrict__ frags = args.frags;
  const float* __restrict__ factors = args.factors;
  const SlotTable table = args.table;
  const half_t* __restrict__ w = args.w;
  const half_t* base = args.base;
  half_t* out = args.out;
  const int C = args.C, R = args.R, L = args.L, slots = args.slots, group = args.group;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, lq = lane >> 4;
  const int blocks = (C + 511) >> 9;
  const int c0 = (block % blocks) * 512 + wave * 128;
  const int c = c0 + 8 * lr;
  const int s0 = (block / blocks) * group;
  if (c0 >= C) return;
  const int ns = min(group, slots - s0);
  // lane l: slot s0 + l
  const int2 meta = lane < ns ? table.meta[s0 + lane] : int2{-1, 0};
  const uint4 far = lane < ns ? reinterpret_cast<const uint4*>(args.wide)[s0 + lane] : uint4{0, 0, 0, 0};
  const uint32_t wide = far.x | (F > 1 ? far.y : 0) | (F > 2 ? far.z : 0) | (F > 3 ? far.w : 0);   // a bit per row
  auto wide_of = [&](int i, int g) { return static_cast<uint32_t>(__builtin_amdgcn_readlane(wide, i)) >> (16 * g) & 0xFFFFu; };
  half8_t wf[F][8];
  auto load_base = [&](StreamRows<F, P>& o) {
    if constexpr (BASE) {
      const half_t* b = base + min(c, C - 8);
      o.y[0] = *reinterpret_cast<const uint4*>(b + static_cast<size_t>(o.row.x) * C);
      o.y[1] = *reinterpret_cast<const uint4*>(b + static_cast<size_t>(o.row.y) * C);
      o.y[2] = *reinterpret_cast<const uint4*>(b + static_cast<size_t>(o.row.z) * C);
      o.y[3] = *reinterpret_cast<const uint4*>(b + static_cast<size_t>(o.row.w) * C);
    }
  };
  auto leave = [&](const StreamRows<F, P>& o, const float4_t (&acc)[8], float4_t factor, uint32_t which) {   // a bit per row
    const int rows[4] = {o.row.x, o.row.y, o.row.z, o.row.w};
    which = c < C ? which >> (4 * lq) : 0;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const half8_t v = expand_result<true>(acc, r, BASE ? o.y[r] : uint4{0, 0, 0, 0}, factor[r]);
      if (which >> r & 1) store_past_l2(out + static_cast<size_t>(rows[r]) * C + c, v);
    }
  };
  auto first_rows = [](int count) { return count < 16 ? (1u << count) - 1u : 0xFFFFu; };   // count > 0

  for (int i = 0; i < ns;) {
    const int adapter = __builtin_amdgcn_readlane(meta.x, i);
    const int count = __builtin_amdgcn_readlane(meta.y, i);
    if (count == 0 || adapter == L) {
      if (count > 0 && base != out)
        for (int m = lq; m < count; m += 4) {
          const size_t at = static_cast<size_t>(table.rows[(s0 + i) * kSlotRows + m]) * C;
          if (c < C) *reinterpret_cast<uint4*>(out + at + c) = BASE ? *reinterpret_cast<const uint4*>(base + at + c) : uint4{0, 0, 0, 0};
        }
      ++i;
      continue;
    }
    // the run: slots i .. end - 1 of the same adapter, all but the last full
    const uint64_t other = __ballot(meta.x != adapter || meta.y == 0) >> i;
    const int end = other ? i + __builtin_ctzll(other) : 64;
    const int last = __builtin_amdgcn_readlane(meta.y, end - 1);
    const int n = 2 * (end - i - 1) + ((last + 15) >> 4);            // row groups
    const int total = 32 * (end - i - 1) + last;                      // rows
    load_expand_weights<F, PACKED, TRANS, true>(w + static_cast<size_t>(adapter) * R * C, c0, C, R, lane, wf);
    const int g0 = 2 * (s0 + i);
    auto load = [&](int g, int4 row, StreamRows<F, P>& o) {   // g < n
      o.row = row;
      o.factor = *reinterpret_cast<const float4_t*>(factors + (g0 + g) * 16 + 4 * lq);
      const half8_t* f8 = reinterpret_cast<const half8_t*>(frags) + static_cast<size_t>(g0 + g) * F * P * 64 + lane;
#pragma unroll
      for (int f = 0; f < F; ++f)
#pragma unroll
        for (int p = 0; p < P; ++p) o.h[f][p] = f8[(f * P + p) * 64];
      load_base(o);
    };
    auto finish = [&](int g, const StreamRows<F, P>& o) {
      float4_t acc[8] = {};
#pragma unroll
      for (int f = 0; f < F; ++f) expand_products<P, true>(wf[f], o.h[f], acc);
      leave(o, acc, o.factor, first_rows(total - 16 * g) & ~wide_of(i + (g >> 1), g & 1));   // wide ones: below
    };
    // rows are looked up D groups ahead of their loads
    auto row_of = [&](int g) {
      return *reinterpret_cast<const int4*>(table.rows + (g0 + min(g, n - 1)) * 16 + 4 * lq);
    };
    StreamRows<F, P> ring[D];
    int4 ahead[D];
#pragma unroll
    for (int d = 0; d < D; ++d) ahead[d] = row_of(d);
#pragma unroll
    for (int d = 0; d < D; ++d) {
      load(min(d, n - 1), ahead[d], ring[d]);
      ahead[d] = row_of(d + D);
    }
    int g = 0;
    for (; g + 2 * D <= n; g += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        finish(g + d, ring[d]);
        load(g + d + D, ahead[d], ring[d]);
        ahead[d] = row_of(g + d + 2 * D);
      }
    }
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (g + d < n) finish(g + d, ring[d]);
      if (g + d + D < n) load(g + d + D, ahead[d], ring[d]);
    }
#pragma unroll
    for (int d = 0; d < D; ++d)
      if (g + d + D < n) finish(g + d + D, ring[d]);
    i = end;
  }

  // Rows in fp32 (weights read again, so that the loop above keeps its registers).
  for (uint64_t left = __ballot(wide != 0 && meta.y > 0 && meta.x != L); left; left &= left - 1) {
    const int i = __builtin_ctzll(left);
    const int adapter = __builtin_amdgcn_readlane(meta.x, i);
    load_expand_weights<F, PACKED, TRANS, true>(w + static_cast<size_t>(adapter) * R * C, c0, C, R, lane, wf);
    const float si = args.scaling ? args.scaling[adapter] : 1.0f;
#pragma unroll 1
    for (int g = 0; g < 2; ++g) {
      if (!wide_of(i, g)) continue;
      const int32_t* rows = table.rows + (s0 + i) * kSlotRows + 16 * g;
      StreamRows<F, P> o;
      o.row = *reinterpret_cast<const int4*>(rows + 4 * lq);
      load_base(o);
      float v[F][8];
      load_ranks<F, PACKED>(args.h + static_cast<size_t>(rows[lr]) * R, R, lq, v);
      // converted anew for each group: in fp32 the weights would not fit the registers
#pragma unroll
      for (int f = 0; f < F; ++f)
#pragma unroll
        for (int t = 0; t < 8; ++t) asm volatile("" : "+v"(wf[f][t]));
      float4_t acc[8];
      expand_products_fp32<F, PACKED, true>(wf, v, lq, acc);
      leave(o, acc, float4_t{si, si, si, si}, first_rows(__builtin_amdgcn_readlane(meta.y, i) - 16 * g) & wide_of(i, g));
    }
  }
}

template <int F, bool PACKED, bool TRANS, bool BASE, int D>
__global__ __launch_bounds__(256, F <= 2 ? 2 : 1) void lora_stream_kernel(StreamArgs args) {
  stream_rows<F, PACKED, TRANS, BASE, D>(args, blockIdx.x);
}

// --- outer: grad_i[c][j] = s_i sum over the rows of adapter i of x[m][c] h[m][j] ----------
//
// A wavefront sums 128 channels x 16 NT ranks over slots of 32 rows; the wavefronts of a
// workgroup take turns along the slots and are added in LDS in a fixed order.  Lane (r, q)
// loads 8 channels (octet r) of its 8 rows (8 q ..) and transposes the 8 x 8 block in
// registers, so that x goes from memory to the MFMA operand without LDS; the next slot's
// rows are in flight meanwhile.  The split h comes as ready operands.
// The products of a slot are summed from zero and join the sums in fp32, times the unit of their
// slot and rank.  A slot whose operands are not whole (negative units; values that lie more than 2^16
// apart within a rank and take more than two terms) is multiplied in fp32 instead, from the summed
// h, at 8 times the MFMA cycles.  Where there are none: training step 291 -> 294 us, backward of 2048
// rows 40.1 -> 40.6 us, the other backward passes within 1%, against one power of two for all ranks
// of a slot and sums in units of the largest slot's.
// A slot's missing rows repeat its first one against zero operands.
// Q8: x is an 8-bit checkpoint, expanded after the transpose (which then moves bytes).
// CMAJOR: gradient [L][C][R] (channels are MFMA rows), else [L][R][C].
// Few channels leave compute units idle, so the slots are dealt to `parts` workgroups (decoded
// from the block after its channels and block of ranks), each with a gradient of its own, added by
// lora_sum_parts_kernel.
template <int NT, bool Q8, bool CMAJOR>
struct OuterSlot {
  uint4 v[8];              // 8 rows of 8 channels (Q8: the codes in x and y)
  uint32_t s2[Q8 ? 4 : 1]; // scales of rows 2 i, 2 i + 1
  half8_t h[NT][2];        // hi and lo operands
  float unit[NT][CMAJOR ? 1 : 4];   // of the ranks of this lane's sums
};

struct OuterArgs {
  const half_t* x;          // or codes and scales (Q8)
  const uint8_t* codes;
  const half_t* xs;
  int gshift;
  const half_t* frags;
  const float* units;
  const float* h;           // [M][R], summed
  const float* scaling;
  RowPlan plan;
  float* grad;
  int C, R, parts;
  int row_waves;            // 4: 128 channels per workgroup; 1: 128 per wavefront
};

// Workgroup `block` of columns x parts x rank blocks x adapters, D slots in flight per
// wavefront.  red: outer_lds(NT, W) entries of LDS.
template <int NT, int W, int D, bool Q8, bool CMAJOR>
__device__ __forceinline__ void outer_sums(const OuterArgs& args, int block, float4_t* red) {
  const half_t* __restrict__ x = args.x;
  const uint8_t* __restrict__ codes = args.codes;
  const half_t* __restrict__ xs = args.xs;
  const half_t* __restrict__ frags = args.frags;
  const float* __restrict__ units = args.units;
  const float* __restrict__ scaling = args.scaling;
  const RowPlan plan = args.plan;
  float* __restrict__ grad = args.grad;
  const int C = args.C, R = args.R, parts = args.parts, gshift = args.gshift;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lq = lane >> 4;
  // Neighbouring workgroups go to different XCDs (8, in turn).  Where there are several blocks
  // of ranks, eight blocks of channels are followed by their further blocks of ranks, which
  // thus find x in the same L2.
  const int ranks = (R + 16 * NT - 1) / (16 * NT);
  const int row_waves = args.row_waves, width = 128 * W / row_waves;   // channels per workgroup
  int col, t0 = 0;
  if (ranks == 1) {
    const int cols = (C + width - 1) / width;
    col = block % cols;
    block /= cols;
  } else {
    const int eights = (C + 8 * width - 1) / (8 * width);
    col = block & 7;
    block >>= 3;
    t0 = (block % ranks) * NT;
    block /= ranks;
    col += 8 * (block % eights);
    block /= eights;
  }
  const int part = block % parts;
  const int ad = block / parts;
  const int c_block = col * width;
  if (c_block >= C) return;
  const int row_wave = row_waves == 1 ? 0 : wave;
  const int c0 = c_block + (row_waves == 1 ? 128 * wave : 0);
  const int NTT = (R + 15) >> 4;   // fragments per slot
  // slots of the adapter: [first_slot, first_slot + n); positions lo .. hi - 1
  const int lo = plan.index ? plan.off[ad] : 0;
  const int hi = plan.index ? plan.off[ad + 1] : ad == 0 ? plan.M : 0;   // no index: all rows are adapter 0's
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
  auto load = [&](int k, OuterSlot<NT, Q8, CMAJOR>& o) {
    const int slot = first_slot + min(k, n - 1);
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
      const float* u = units + (static_cast<size_t>(slot) * NTT + tt) * 16;
      if constexpr (CMAJOR) {
        o.unit[t][0] = u[lr];
      } else {
        const float4_t u4 = *reinterpret_cast<const float4_t*>(u + 4 * lq);
#pragma unroll
        for (int r = 0; r < 4; ++r) o.unit[t][r] = u4[r];
      }
    }
  };

  float4_t acc[8][NT] = {};
  // Slots that are not whole are left for later: bit i for this wavefront's slots from i <<
  // left_shift on, 64 such runs at most.
  uint64_t left = 0;
  int left_shift = 0;
  auto add = [&](int k, const OuterSlot<NT, Q8, CMAJOR>& o) {
    bool whole = true;   // the 16 units of a fragment have one sign
#pragma unroll
    for (int t = 0; t < NT; ++t) whole &= __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, o.unit[t][0])) >= 0;
    if (!whole) {
      left |= 1ull << (k >> left_shift);
      return;
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
      for (int t = 0; t < NT; ++t) {
        float4_t v = {};
#pragma unroll
        for (int p = 0; p < 2; ++p)
          v = CMAJOR ? __builtin_amdgcn_mfma_f32_16x16x32_f16(xf, o.h[t][p], v, 0, 0, 0)
                     : __builtin_amdgcn_mfma_f32_16x16x32_f16(o.h[t][p], xf, v, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[c][t][r] = fmaf(v[r], o.unit[t][CMAJOR ? 0 : r], acc[c][t][r]);
      }
    }
  };
  // A slot in fp32, four rows at a time: step i takes row 8 q + i of every quarter q.
  auto add_fp32 = [&](int k) {
    bool whole = true;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float u = units[(static_cast<size_t>(first_slot + k) * NTT + min(t0 + t, NTT - 1)) * 16];
      whole &= __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, u)) >= 0;
    }
    if (whole) return;
    const int p0 = lo + k * kSlotRows;
#pragma unroll 4
    for (int i = 0; i < 8; ++i) {
      const bool in = p0 + 8 * lq + i < hi;
      const int p = in ? p0 + 8 * lq + i : p0;
      const size_t m = plan.index ? plan.perm[p] : p;
      half8_t xv;
      if constexpr (Q8) {
        const uint2 c = *reinterpret_cast<const uint2*>(codes + m * C + cc);
        const half_t s = xs[m * G + (cc >> gshift)];
        xv = act_values(c, half2_t{s, s});
      } else {
        xv = *reinterpret_cast<const half8_t*>(x + m * C + cc);
      }
      float h[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int j = 16 * (t0 + t) + lr;
        h[t] = in && j < R ? args.h[m * R + j] : 0.0f;
      }
#pragma unroll
      for (int c = 0; c < 8; ++c)
#pragma unroll
        for (int t = 0; t < NT; ++t)
          acc[c][t] = CMAJOR ? __builtin_amdgcn_mfma_f32_16x16x4f32(static_cast<float>(xv[c]), h[t], acc[c][t], 0, 0, 0)
                             : __builtin_amdgcn_mfma_f32_16x16x4f32(h[t], static_cast<float>(xv[c]), acc[c][t], 0, 0, 0);
    }
  };

  if (n > 0) {
    OuterSlot<NT, Q8, CMAJOR> ring[D];
    const int first = part * row_waves + row_wave, stride = parts * row_waves;
    const int mine = first < n ? (n - first + stride - 1) / stride : 0;   // slots of this wavefront
    auto slot_of = [&](int k) { return first + k * stride; };
    while (mine > 64 << left_shift) ++left_shift;
    find_rows(slot_of(0));
#pragma unroll
    for (int d = 0; d < D; ++d) {
      load(slot_of(d), ring[d]);
      find_rows(slot_of(d + 1));
    }
    // The main loop reloads a stage as soon as it is used; the tail loads only what is left.
    int k = 0;
    for (; k + 2 * D <= mine; k += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        add(k + d, ring[d]);
        load(slot_of(k + d + D), ring[d]);
        find_rows(slot_of(k + d + D + 1));
      }
    }
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (k + d < mine) add(k + d, ring[d]);
      if (k + d + D < mine) {
        load(slot_of(k + d + D), ring[d]);
        find_rows(slot_of(k + d + D + 1));
      }
    }
#pragma unroll
    for (int d = 0; d < D; ++d)
      if (k + d + D < mine) add(k + d + D, ring[d]);
    while (left) {
      const int at = __builtin_ctzll(left) << left_shift;
      left &= left - 1;
#pragma unroll 1
      for (k = at; k < min(mine, at + (1 << left_shift)); ++k) add_fp32(slot_of(k));
    }
  }

  // The sums are collected in LDS in the order of the gradient and leave as
  // whole rows: the workgroup's 128 channels, one channel fragment of all wavefronts at a
  // time, or the 128 channels of one wavefront after the other.
  const float si = n == 0 ? 0.0f : scaling ? scaling[ad] : 1.0f;
  float* sums = reinterpret_cast<float*>(red + W * NT * 64);   // [128][16 NT + 4] or [16 NT][128 + 4]
  constexpr int ld = CMAJOR ? 16 * NT + 4 : 128 + 4;
  float* g = grad + (static_cast<size_t>(part) * plan.L + ad) * R * C;
  auto collect = [&](int c, int j0, int l, const float4_t& v) {   // lane l's sums of fragment c
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int ch = CMAJOR ? 8 * (4 * (l >> 4) + r) + c : 8 * (l & 15) + c;
      const int j = CMAJOR ? j0 + (l & 15) : j0 + 4 * (l >> 4) + r;
      sums[CMAJOR ? ch * ld + j : j * ld + ch] = si * v[r];
    }
  };
  auto leave = [&](int cb) {   // channels cb .. cb + 127
    const int nj = min(16 * NT, R - 16 * t0), nc = min(128, C - cb);   // both multiples of 8
    const int quads = (CMAJOR ? nj : nc) >> 2, lines = CMAJOR ? nc : nj;
    for (int i = tid; i < quads * lines; i += 64 * W) {
      const int line = i / quads, q = i % quads;
      const float4_t v = *reinterpret_cast<const float4_t*>(sums + line * ld + 4 * q);
      float* o = CMAJOR ? g + static_cast<size_t>(cb + line) * R + 16 * t0 : g + static_cast<size_t>(16 * t0 + line) * C + cb;
      *reinterpret_cast<float4_t*>(o + 4 * q) = v;
    }
  };
  if (row_waves == 1) {
    for (int turn = 0; turn < W; ++turn) {
      if (c_block + 128 * turn >= C) break;
      if (wave == turn)
#pragma unroll
        for (int c = 0; c < 8; ++c)
#pragma unroll
          for (int t = 0; t < NT; ++t) collect(c, 16 * t, lane, acc[c][t]);
      __syncthreads();
      leave(c_block + 128 * turn);
      __syncthreads();
    }
    return;
  }
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t) red[(wave * NT + t) * 64 + lane] = acc[c][t];
    __syncthreads();
    for (int i = tid; i < NT * 64; i += 64 * W) {
      float4_t v = red[i];
      for (int w = 1; w < W; ++w) v += red[w * NT * 64 + i];
      collect(c, 16 * (i / 64), i & 63, v);
    }
  }
  __syncthreads();
  leave(c_block);
}

// Entries of LDS that outer_sums needs (the larger of its two gradient layouts).
constexpr int outer_lds(int NT, int W) {
  const int by_channel = 128 * (16 * NT + 4), by_rank = 16 * NT * (128 + 4);
  return W * NT * 64 + (by_channel > by_rank ? by_channel : by_rank) / 4;
}

// dB and dA in one launch: the workgroups of the second fill what the first leaves idle.
template <bool Q8>
__global__ __launch_bounds__(256, 2) void lora_outers_kernel(OuterArgs b, int b_blocks, OuterArgs a) {
  __shared__ float4_t red[outer_lds(2, 4)];
  const int block = blockIdx.x;
  if (block < b_blocks) outer_sums<2, 4, 2, false, true>(b, block, red);
  else outer_sums<2, 4, 2, Q8, false>(a, block - b_blocks, red);
}

// The three products of the backward pass in one launch: their workgroups fill the GPU
// together (the outer products alone have one per 128 channels and block of ranks), and two
// launches fall away.  HBM-bound where it is large: 4096 rows, K = 8192 in 8 bits, N = 28672, rank
// 64: 98 us for 459 MB, 4.7 TB/s (240 training steps in a row; 106 us in the first dozen).  Workgroups: dB, then dA, then dx (F fragments of 32 ranks).
template <int NT, int F, bool Q8, bool DX, bool BASE>
__global__ __launch_bounds__(256, 2) void lora_products_kernel(OuterArgs b, int b_blocks, OuterArgs a, int a_blocks,
                                                               StreamArgs dx) {
  __shared__ float4_t red[outer_lds(NT, 4)];
  const int block = blockIdx.x;
  if (block < b_blocks) {
    outer_sums<NT, 4, 2, false, true>(b, block, red);
  } else if (block < b_blocks + a_blocks) {
    outer_sums<NT, 4, 2, Q8, false>(a, block - b_blocks, red);
  } else {
    if constexpr (DX) stream_rows<F, NT == 1, true, BASE, 2>(dx, block - b_blocks - a_blocks);
  }
}

// out = sum of the parts, in order; both gradients in one launch (blockIdx.y), 4 us.
struct PartsTask {
  const float4_t* parts;
  float4_t* out;
  size_t quads;
  int count;
};

__global__ __launch_bounds__(256) void lora_sum_parts_kernel(PartsTask t0, PartsTask t1) {
  const PartsTask t = blockIdx.y == 0 ? t0 : t1;
  const size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= t.quads) return;
  float4_t v = t.parts[i];
  for (int p = 1; p < t.count; ++p) v += t.parts[p * t.quads + i];
  t.out[i] = v;
}

}  // namespace w4a16
