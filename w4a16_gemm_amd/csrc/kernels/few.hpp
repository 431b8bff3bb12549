// Products grouped by expert for few rows each (decode): y^T = W^_e x^T with the weights as
// the MFMA's A operand (16 outputs) and up to 16 rows of an expert as its B operand.
//
// Bound by the stream of the used experts' codes, so the kernel is built around it:
//  * One launch and no plan before it: the experts of up to kFewSlots slots are counted by
//    every workgroup itself, while its threads would wait for memory anyhow.
//  * The units of work are 16 outputs of a row tile (up to 16 rows of one expert), over all
//    tiles; every workgroup takes an equal run of them, whatever the groups' sizes, the
//    workgroups of one XCD neighbouring runs.
//  * The wavefronts of a workgroup split K: wavefront w holds the activations of T steps of
//    128 channels in registers and streams its part of the codes straight to registers, each
//    step's slot refilled for the next unit as soon as it is used.  Lane (r, q) loads 16 bytes
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

struct FewLds {
  int32_t expert[kFewSlots];
  int32_t count[kMaxExperts];
  int32_t tile0[kMaxExperts + 1];   // first row tile of every expert
  int32_t slot[16];                 // of the current tile
  int32_t rows, current;
};

constexpr size_t few_lds(int waves) { return sizeof(FewLds) + static_cast<size_t>(kFewBatch) * waves * 1024; }

// The slots of one 16-row tile into lds.slot / lds.rows, its expert into lds.current.  All
// threads; ends with a barrier.
__device__ __forceinline__ void find_few_tile(FewLds& lds, int S, int E, int tile, int tid, int threads) {
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
}

// x: row of slot s is s / T (by_slot: s).
template <int STEPS, int BITS>
__global__ __launch_bounds__(1024) void experts_few_kernel(const half_t* __restrict__ x, int by_slot, int T,
                                                           const int32_t* __restrict__ index, int S, int E, Layers layers,
                                                           int chunks, half_t* __restrict__ y) {
  constexpr int NQ = BITS / 4;          // 16-byte loads per lane and step
  constexpr int PER = 32 / BITS;        // channels per word
  extern __shared__ __align__(16) unsigned char smem[];
  FewLds& lds = *reinterpret_cast<FewLds*>(smem);
  float* red = reinterpret_cast<float*>(smem + sizeof(FewLds));   // [unit of the batch][wave][16 rows][16 outputs]
  const int tid = threadIdx.x, threads = blockDim.x, waves = threads >> 6;
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lq = lane >> 4;
  const int N = layers.N, K = layers.K;
  const int blocks = (N + 15) >> 4;   // units per row tile

  // experts of the slots, row tiles of the experts
  for (int e = tid; e < E; e += threads) lds.count[e] = 0;
  __syncthreads();
  for (int s = tid; s < S; s += threads) {
    const int e = index[s];
    const bool valid = e >= 0 && e < E;
    lds.expert[s] = valid ? e : -1;
    if (valid) atomicAdd(&lds.count[e], 1);
  }
  __syncthreads();
  if (wave == 0) {
    int carry = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const int e = e0 + lane;
      const int tiles = e < E ? (lds.count[e] + 15) >> 4 : 0;
      int sum = tiles;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(sum, d);
        if (lane >= d) sum += o;
      }
      if (e < E) lds.tile0[e] = carry + sum - tiles;
      carry += __shfl(sum, 63);
    }
    if (lane == 0) lds.tile0[E] = carry;
  }
  __syncthreads();
  const int units = lds.tile0[E] * blocks;
  const int per = (units + gridDim.x - 1) / gridDim.x;
  int u = min(units, xcd_block(blockIdx.x, gridDim.x) * per);
  const int u_end = min(units, u + per);

  // one unit's operands of this lane: codes, scale and zero point of every step
  uint4 cw[STEPS][NQ];
  uint32_t sc[STEPS], zw[STEPS];
  Layers l = layers;
  const uint32_t pitch = static_cast<uint32_t>(K) * BITS / 8;
  __amdgpu_buffer_rsrc_t codes = stream_rsrc(layers.qw, 0);
  auto channel = [&](int c, int t) { return ((c * waves + wave) * STEPS + t) * 128 + 32 * lq; };
  auto load_step = [&](int b, int c, int t) {
    const int n = min(16 * b + lr, N - 1), k = min(channel(c, t), K - 32), g = k >> l.gshift;
    const uint32_t at = static_cast<uint32_t>(n) * pitch + static_cast<uint32_t>(k) * BITS / 8;
#pragma unroll
    for (int q = 0; q < NQ; ++q) cw[t][q] = load_buffer16(codes, at + 16u * q);
    sc[t] = __builtin_bit_cast(uint16_t, l.scales[static_cast<size_t>(g) * N + n]);
    zw[t] = *l.zeros.at(static_cast<size_t>(g) * (N / PER) + n / PER);
  };

  while (u < u_end) {
    const int tile = u / blocks;
    find_few_tile(lds, S, E, tile, tid, threads);
    const int rows = lds.rows, last = min(u_end, (tile + 1) * blocks);
    l = layers.at<BITS>(lds.current);
    codes = stream_rsrc(l.qw, static_cast<uint32_t>(N) * pitch);
#pragma unroll
    for (int t = 0; t < STEPS; ++t) load_step(u - tile * blocks, 0, t);
    const int m = lds.slot[min(lr, rows - 1)];
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
    if (chunks == 1) load_x(0);
    for (; u < last; u += kFewBatch) {
      const int batch = min(kFewBatch, last - u), b0 = u - tile * blocks;
      for (int c = 0; c < chunks; ++c) {
        if (chunks > 1) load_x(c);
        for (int i = 0; i < batch; ++i) {
          // the unit after this one: of this batch, of its next chunk, of the next batch
          int nb = b0 + i + 1, nc = c;
          if (i + 1 == batch) {
            nc = c + 1 < chunks ? c + 1 : 0;
            if (c + 1 < chunks) nb = b0;
          }
          nb = min(nb, blocks - 1);
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
              if constexpr (BITS == 4) {
                w[j] = dequant_word(j == 0 ? cw[t][0].x : j == 1 ? cw[t][0].y : j == 2 ? cw[t][0].z : cw[t][0].w, dc);
              } else {
                const uint4 q = cw[t][j >> 1];
                const half4_t lo = dequant_word8((j & 1) ? q.z : q.x, dc), hi = dequant_word8((j & 1) ? q.w : q.y, dc);
                w[j] = half8_t{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
              }
            }
            load_step(nb, nc, t);
            a0 = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[0], xr[t][0], a0, 0, 0, 0);
            a1 = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[1], xr[t][1], a1, 0, 0, 0);
            a0 = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[2], xr[t][2], a0, 0, 0, 0);
            a1 = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[3], xr[t][3], a1, 0, 0, 0);
          }
          // lane (r, q) holds outputs 4 q + 0..3 of row r
          float4_t* mine = reinterpret_cast<float4_t*>(red + (i * waves + wave) * 256 + lr * 16 + 4 * lq);
          float4_t s = a0 + a1;
          if (c > 0) s += *mine;
          *mine = s;
        }
      }
      __syncthreads();
      for (int o = tid; o < batch * rows * 16; o += threads) {
        const int i = o / (rows * 16), at = o % (rows * 16), n = 16 * (b0 + i) + (at & 15);
        float s = 0.f;
        for (int w = 0; w < waves; ++w) s += red[(i * waves + w) * 256 + at];
        if (n < N) y[static_cast<size_t>(lds.slot[at >> 4]) * N + n] = static_cast<half_t>(s);
      }
      __syncthreads();
    }
    u = last;
  }

  // slots without an expert
  for (int s = blockIdx.x; s < S; s += gridDim.x)
    if (lds.expert[s] < 0)
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
