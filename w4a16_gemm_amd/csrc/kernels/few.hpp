// Products grouped by expert for few rows each (decode): y^T = W^_e x^T with the weights as
// the MFMA's A operand (16 outputs) and up to 16 rows of an expert as its B operand.
//
// Bound by the stream of the used experts' codes, so the kernel is built around it:
//  * One launch and no plan before it: the experts of up to kFewSlots slots are counted by
//    every workgroup itself, of up to 64 slots by every wavefront.
//  * The units of work are 16 outputs of a row tile (up to 16 rows of one expert), over all
//    tiles; every workgroup takes an equal run of them, whatever the groups' sizes, the
//    workgroups of one XCD neighbouring runs.
//  * The wavefronts of a workgroup split K: wavefront w holds the activations of T steps of
//    128 channels in registers and streams its part of the codes straight to registers, each
//    step's slot refilled for the next unit as soon as it is used (two units ahead are no
//    faster: two experts of 14336 outputs of 4096 channels for one token 17.8 us for 16.9).  Lane (r, q) loads 16 bytes
//    (32 at 8 bits) of output r: channels [128 t + 32 q, +32), one group, whose words are its
//    operands of four MFMAs.  Rows longer than 128 x 16 T channels are walked in `chunks`.
//  * Partial tiles stay in LDS, a slot per wavefront and unit: the wavefronts run through
//    kFewBatch units without a barrier, then the slots are summed in a fixed order.
// Weights are binary16((q - Z) S), as in the large tiles.
#pragma once

#include "plan.hpp"

namespace w4a16 {

constexpr int kFewSlots = 512;
constexpr int kFewBatch = 8;

// The partial tiles lie behind it: whole 16-byte accesses.
struct alignas(16) FewLds {
  int32_t expert[kFewSlots];
  int32_t count[kMaxExperts];
  int32_t tile0[kMaxExperts + 1];   // first row tile of every expert
  int32_t slot[16];                 // of the current tile
  int32_t rows, current;
};

template <bool WAVE>
constexpr size_t few_lds(int waves) {
  return (WAVE ? 0 : sizeof(FewLds)) + static_cast<size_t>(kFewBatch) * waves * 1024;
}

// The row tiles of the slots' experts, up to 16 slots of one expert each.  FewPlan<true>: up to
// 64 slots, a slot per lane, made by every wavefront for itself without a barrier, experts in
// the order of their first slots (one token on two experts: 15.3 us in place of 16.8).
template <bool WAVE>
struct FewPlan;

template <>
struct FewPlan<true> {
  int lane, e, tile0, tiles, total;   // of this lane's slot; tiles of all
  int expert, rows, slot;             // the tile found last; lane r < 16: its slot r

  __device__ __forceinline__ FewPlan(unsigned char*, const int32_t* index, int S, int E, int tid, int) : lane(tid & 63) {
    e = lane < S ? index[lane] : -1;
    if (e >= E || e < 0) e = -1;
    int count = 0, before = 0;
    for (int j = 0; j < S; ++j) {
      const bool like = __builtin_amdgcn_readlane(e, j) == e;
      count += like;
      before += like && j < lane;
    }
    tiles = e >= 0 && before == 0 ? (count + 15) >> 4 : 0;
    int sum = tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(sum, d);
      if (lane >= d) sum += o;
    }
    tile0 = sum - tiles;
    total = __builtin_amdgcn_readlane(sum, 63);
  }
  __device__ __forceinline__ void find(int tile, int) {
    const int at = __ffsll(__ballot(tile0 <= tile && tile < tile0 + tiles)) - 1;
    expert = __builtin_amdgcn_readlane(e, at);
    const int from = 16 * (tile - __builtin_amdgcn_readlane(tile0, at));
    const unsigned long long all = __ballot(e == expert);
    const int rank = __popcll(all & ((1ull << lane) - 1)) - from;
    // every lane gives its slot to the lane of its rank; the others' to lane 63
    slot = __builtin_amdgcn_ds_permute((e == expert && rank >= 0 && rank < 16 ? rank : 63) * 4, lane);
    rows = min(16, static_cast<int>(__popcll(all)) - from);
  }
  // r < 16; lanes 0 .. 15 take part
  __device__ __forceinline__ int slot_of(int r) const { return __shfl(slot, r); }
  __device__ __forceinline__ bool empty(int s) const { return __builtin_amdgcn_readlane(e, s) < 0; }
};

// Up to kFewSlots slots, in LDS, experts in their own order.
template <>
struct FewPlan<false> {
  FewLds& lds;
  int S, E, threads, total, expert, rows;

  __device__ __forceinline__ FewPlan(unsigned char* smem, const int32_t* index, int S_, int E_, int tid, int threads_)
      : lds(*reinterpret_cast<FewLds*>(smem)), S(S_), E(E_), threads(threads_) {
    for (int e = tid; e < E; e += threads) lds.count[e] = 0;
    __syncthreads();
    for (int s = tid; s < S; s += threads) {
      const int e = index[s];
      const bool valid = e >= 0 && e < E;
      lds.expert[s] = valid ? e : -1;
      if (valid) atomicAdd(&lds.count[e], 1);
    }
    __syncthreads();
    if (tid < 64) {
      int carry = 0;
      for (int e0 = 0; e0 < E; e0 += 64) {
        const int e = e0 + tid;
        const int tiles = e < E ? (lds.count[e] + 15) >> 4 : 0;
        int sum = tiles;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
          const int o = __shfl_up(sum, d);
          if (tid >= d) sum += o;
        }
        if (e < E) lds.tile0[e] = carry + sum - tiles;
        carry += __shfl(sum, 63);
      }
      if (tid == 0) lds.tile0[E] = carry;
    }
    __syncthreads();
    total = lds.tile0[E];
  }
  // all threads; ends with a barrier
  __device__ __forceinline__ void find(int tile, int tid) {
    for (int e = tid; e < E; e += threads)
      if (lds.tile0[e] <= tile && tile < lds.tile0[e + 1]) lds.current = e;
    __syncthreads();
    if (tid < 64) {
      const int e = lds.current, from = 16 * (tile - lds.tile0[e]);
      int before = 0;
      for (int s0 = 0; s0 < S; s0 += 64) {
        const int s = s0 + tid;
        const bool mine = s < S && lds.expert[s] == e;
        const unsigned long long all = __ballot(mine);
        const int rank = before + __popcll(all & ((1ull << tid) - 1)) - from;
        if (mine && rank >= 0 && rank < 16) lds.slot[rank] = s;
        before += __popcll(all);
      }
      if (tid == 0) lds.rows = min(16, before - from);
    }
    __syncthreads();
    expert = __builtin_amdgcn_readfirstlane(lds.current);
    rows = __builtin_amdgcn_readfirstlane(lds.rows);
  }
  __device__ __forceinline__ int slot_of(int r) const { return lds.slot[r]; }
  __device__ __forceinline__ bool empty(int s) const { return lds.expert[s] < 0; }
};

// x: row of slot s is s / T (by_slot: s).  LONG: rows in more than one chunk; short ones have
// their kernel, whose activations stay in registers and whose loop keeps no addresses of them.
template <int STEPS, int BITS, bool LONG, bool WAVE>
__global__ __launch_bounds__(1024) void experts_few_kernel(const half_t* __restrict__ x, int by_slot, int T,
                                                           const int32_t* __restrict__ index, int S, int E, Layers layers,
                                                           int chunk_count, half_t* __restrict__ y) {
  const int chunks = LONG ? chunk_count : 1;
  constexpr int NQ = BITS / 4;          // 16-byte loads per lane and step
  constexpr int PER = 32 / BITS;        // channels per word
  extern __shared__ __align__(16) unsigned char smem[];
  float* red = reinterpret_cast<float*>(smem + (WAVE ? 0 : sizeof(FewLds)));   // [unit of the batch][wave][16 rows][16 outputs]
  const int tid = threadIdx.x, threads = blockDim.x, waves = threads >> 6;
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lq = lane >> 4;
  const int N = layers.N, K = layers.K;
  const int blocks = (N + 15) >> 4;   // units per row tile

  FewPlan<WAVE> plan(smem, index, S, E, tid, threads);
  const int units = plan.total * blocks;
  const int per = (units + gridDim.x - 1) / gridDim.x;
  int u = min(units, xcd_block(blockIdx.x, gridDim.x) * per);
  const int u_end = min(units, u + per);

  // one unit's operands of this lane: codes, scale and zero point of every step
  uint4 cw[STEPS][NQ];
  uint32_t sc[STEPS], zw[STEPS];
  Layers l = layers;
  const uint32_t pitch = static_cast<uint32_t>(K) * BITS / 8;
  __amdgpu_buffer_rsrc_t codes = stream_rsrc(layers.qw, 0), scales = codes, zeros = codes;
  auto channel = [&](int c, int t) { return ((c * waves + wave) * STEPS + t) * 128 + 32 * lq; };
  // Outputs past the last (N % 16 = 8) read other outputs' values, or zeros past the buffers'
  // ends, and are not stored.
  auto load_step = [&](int b, int c, int t) {
    const uint32_t k = min(channel(c, t), K - 32), g = k >> l.gshift;
#pragma unroll
    for (int q = 0; q < NQ; ++q)
      cw[t][q] = load_buffer16(codes, lr * pitch + k * BITS / 8 + 16u * q + static_cast<uint32_t>(b) * (16 * pitch));
    // past K: the last channels' codes against rows of 0, with the scale 0 that lies behind the buffer,
    // so that no infinite weight meets such a 0
    const uint32_t at = channel(c, t) < K ? g * N + lr : static_cast<uint32_t>(N) * l.G;
    sc[t] = static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(scales, 2 * at + 32 * b, 0, 0));
    zw[t] = __builtin_amdgcn_raw_buffer_load_b32(zeros, l.zeros.sym ? 0 : 4 * (g * (N / PER) + lr / PER) + 64 / PER * b, 0, 0);
  };

  while (u < u_end) {
    const int tile = u / blocks;
    plan.find(tile, tid);
    const int rows = plan.rows, last = min(u_end, (tile + 1) * blocks);
    l = layers.at<BITS>(plan.expert);
    codes = stream_rsrc(l.qw, static_cast<uint32_t>(N) * pitch);
    scales = stream_rsrc(reinterpret_cast<const uint32_t*>(l.scales), 2u * N * l.G);
    zeros = stream_rsrc(l.zeros.words, static_cast<uint32_t>(N) / PER * 4 * l.G);
    // where the loads are, a unit ahead: unit i of a batch from b0 on, chunk c
    int ai = 0, ac = 0, ab0 = u - tile * blocks, abatch = min(kFewBatch, last - u);
    const int end = last - tile * blocks;
    auto advance = [&]() {
      if (++ai < abatch) return;
      ai = 0;
      if (LONG && ++ac < chunks) return;
      ac = 0;
      ab0 += abatch;
      abatch = max(1, min(kFewBatch, end - ab0));
    };
#pragma unroll
    for (int t = 0; t < STEPS; ++t) load_step(ab0, 0, t);
    advance();
    const int m = plan.slot_of(min(lr, rows - 1));
    const half_t* row = x + static_cast<size_t>(by_slot ? m : m / T) * K;
    half8_t xr[STEPS][4];
    auto load_x = [&](int c) {
#pragma unroll
      for (int t = 0; t < STEPS; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = channel(c, t) + 8 * j;
          const half8_t v = *reinterpret_cast<const half8_t*>(row + min(k, K - 8));
          xr[t][j] = lr < rows && k < K ? v : half8_t{};
        }
    };
    load_x(0);
    int b0 = u - tile * blocks, batch = min(kFewBatch, last - u), i = 0, c = 0;
    while (batch > 0) {
      float4_t a0 = {0.f, 0.f, 0.f, 0.f}, a1 = a0;
#pragma unroll
      for (int t = 0; t < STEPS; ++t) {
        uint32_t z;
        if constexpr (BITS == 4)
          z = (l.zeros.word(zw[t]) >> (4 * (lr & 7))) & 0xFu;
        else
          z = (l.zeros.word8(zw[t]) >> (8 * (lr & 3))) & 0xFFu;
        const DequantConsts dc = make_consts(z, __builtin_bit_cast(half_t, static_cast<uint16_t>(sc[t])));
        half8_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 q = cw[t][BITS == 4 ? 0 : j >> 1];
          if constexpr (BITS == 4) {
            w[j] = dequant_word(j == 0 ? q.x : j == 1 ? q.y : j == 2 ? q.z : q.w, dc);
          } else {
            const half4_t lo = dequant_word8((j & 1) ? q.z : q.x, dc), hi = dequant_word8((j & 1) ? q.w : q.y, dc);
            w[j] = half8_t{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
          }
        }
        load_step(min(ab0 + ai, blocks - 1), ac, t);
        a0 = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[0], xr[t][0], a0, 0, 0, 0);
        a1 = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[1], xr[t][1], a1, 0, 0, 0);
        a0 = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[2], xr[t][2], a0, 0, 0, 0);
        a1 = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[3], xr[t][3], a1, 0, 0, 0);
      }
      advance();
      // lane (r, q) holds outputs 4 q + 0..3 of row r
      float4_t* mine = reinterpret_cast<float4_t*>(red + (i * waves + wave) * 256 + lr * 16 + 4 * lq);
      float4_t s = a0 + a1;
      if (LONG && c > 0) s += *mine;
      *mine = s;
      if (++i < batch) continue;
      i = 0;
      if constexpr (LONG) {
        if (++c < chunks) {
          load_x(c);
          continue;
        }
        c = 0;
      }
      __syncthreads();
      for (int o = tid; o < batch * rows * 16; o += threads) {
        const int from = o / (rows * 16), at = o % (rows * 16), n = 16 * (b0 + from) + (at & 15);
        const int slot = plan.slot_of(at >> 4);
        float sum = 0.f;
        for (int w = 0; w < waves; ++w) sum += red[(from * waves + w) * 256 + at];
        if (n < N) y[static_cast<size_t>(slot) * N + n] = static_cast<half_t>(sum);
      }
      __syncthreads();
      b0 += batch;
      batch = min(kFewBatch, end - b0);
      if (LONG && batch > 0) load_x(0);
    }
    u = last;
  }

  // slots without an expert
  for (int s = blockIdx.x; s < S; s += gridDim.x)
    if (plan.empty(s))
      for (int n = 8 * tid; n < N; n += 8 * threads)
        *reinterpret_cast<half8_t*>(y + static_cast<size_t>(s) * N + n) = half8_t{};
}

// Act order: out[s] = the row of slot s in the stored channel order of its expert.
__global__ __launch_bounds__(256) void gather_rows_kernel(const half_t* __restrict__ x, const int32_t* __restrict__ index,
                                                          int E, Layers layers, int T, half_t* __restrict__ out) {
  const int s = blockIdx.x, K = layers.K, e = index[s];
  if (e < 0 || e >= E) return;
  const int32_t* at = layers.order(e);
  const half_t* row = x + static_cast<size_t>(s / T) * K;
  for (int i = 8 * threadIdx.x; i < K; i += 8 * 256) {
    half8_t v;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = row[min(static_cast<uint32_t>(at[i + j]), static_cast<uint32_t>(K - 1))];
    *reinterpret_cast<half8_t*>(out + static_cast<size_t>(s) * K + i) = v;
  }
}

}  // namespace w4a16
