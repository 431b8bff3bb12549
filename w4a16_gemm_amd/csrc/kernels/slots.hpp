// Slots grouped by expert, by one workgroup:
//  * each wavefront counts the experts of its own run of slots in an LDS histogram of its
//    own; a scan over the wavefronts of every expert and over the experts gives every
//    wavefront the place of its first slot of every expert;
//  * the second pass ranks the 64 slots of a load among themselves by ballots over the bits
//    of the expert's number (10 at most), so that the order is stable and does not depend on
//    timing.
// Slots without an expert come last, in no tile.  Bound by the latency of the two passes: 8 loads of 64
// slots per wavefront are in flight at once.  And the channel orders of act order.
#pragma once

#include "plan.hpp"

namespace w4a16 {

// Slots with index outside [0, limit) have no expert; index NULL: expert 0 for every slot.
// E == limit, or E == 1: every slot with an index inside belongs to expert 0.
__global__ __launch_bounds__(kPlanThreads) void plan_slots_kernel(const int32_t* __restrict__ index, int S, int E,
                                                                  int limit, int height, SlotPlan plan) {
  extern __shared__ int32_t hist[];   // [kPlanWaves][E + 1]
  __shared__ int32_t first[kMaxExperts + 2];
  __shared__ int32_t tile0[kMaxExperts + 2];
  __shared__ int32_t wave_sum[kPlanWaves][2];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int bins = E + 1;
  for (int i = tid; i < kPlanWaves * bins; i += kPlanThreads) hist[i] = 0;
  __syncthreads();

  constexpr int U = 8;
  const int run = ((S + kPlanWaves - 1) / kPlanWaves + 63) / 64 * 64;
  const int begin = min(static_cast<int64_t>(S), static_cast<int64_t>(wave) * run);
  const int end = min(static_cast<int64_t>(S), static_cast<int64_t>(begin) + run);
  int32_t* mine = hist + wave * bins;
  auto expert_of = [&](int s) {
    if (s >= end) return -1;   // no slot
    const int e = index ? index[s] : 0;
    return e < 0 || e >= limit ? E : E == 1 ? 0 : e;
  };
  for (int s0 = begin; s0 < end; s0 += 64 * U) {
    int e[U];
#pragma unroll
    for (int u = 0; u < U; ++u) e[u] = expert_of(min(s0 + 64 * u, end) + lane);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (e[u] >= 0) atomicAdd(&mine[e[u]], 1);
  }
  __syncthreads();

  // per expert: the wavefronts' counts become places inside the expert's slots
  int count = 0, tiles = 0;
  if (tid < bins) {
    for (int w = 0; w < kPlanWaves; ++w) {
      const int c = hist[w * bins + tid];
      hist[w * bins + tid] = count;
      count += c;
    }
    if (tid < E) tiles = count / height + (count % height != 0);
  }
  // exclusive scan of (count, tiles) over the experts
  int pc = count, pt = tiles;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int c = __shfl_up(pc, d), t = __shfl_up(pt, d);
    if (lane >= d) pc += c, pt += t;
  }
  if (lane == 63) wave_sum[wave][0] = pc, wave_sum[wave][1] = pt;
  __syncthreads();
  int oc = 0, ot = 0;
  for (int w = 0; w < wave; ++w) oc += wave_sum[w][0], ot += wave_sum[w][1];
  pc += oc - count;
  pt += ot - tiles;
  if (tid < bins) first[tid] = pc, tile0[tid] = pt;
  if (tid == E) {
    plan.counts[0] = pt + tiles;
    plan.counts[1] = pc;
  }
  if (tid < bins)
    for (int i = 0; i < tiles; ++i) {
      RowTile t;
      t.expert = tid;
      t.first = pc + i * height;
      t.rows = min(height, count - i * height);
      t.height = rest_height(t.rows, height);
      t.panel_first = pt + i / kPanelTiles * kPanelTiles;
      t.panel_tiles = min(kPanelTiles, pt + tiles - t.panel_first);
      t.pad[0] = t.pad[1] = 0;
      plan.tiles[pt + i] = t;
    }
  __syncthreads();

  const int bits = 32 - __clz(E);
  for (int s0 = begin; s0 < end; s0 += 64 * U) {
    int e[U];
#pragma unroll
    for (int u = 0; u < U; ++u) e[u] = expert_of(min(s0 + 64 * u, end) + lane);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      unsigned long long same = __ballot(e[u] >= 0);
      for (int b = 0; b < bits; ++b) {
        const unsigned long long set = __ballot((e[u] >> b) & 1);
        same &= (e[u] >> b) & 1 ? set : ~set;
      }
      const int rank = __popcll(same & ((1ull << lane) - 1));
      if (e[u] >= 0) {
        const int within = mine[e[u]] + rank;
        plan.order[first[e[u]] + within] = s0 + 64 * u + lane;
        if (plan.tile_of) plan.tile_of[s0 + 64 * u + lane] = tile0[e[u]] + within / height;
      }
      __builtin_amdgcn_wave_barrier();
      if (e[u] >= 0 && rank == 0) mine[e[u]] += __popcll(same);
      __builtin_amdgcn_wave_barrier();
    }
  }
}

// Act order: the rows of the valid slots, each in the stored channel order of its expert:
// out[p][i] = x[order[p] / T][channel at stored position i].  Eight channels per thread.
__global__ __launch_bounds__(256) void gather_slots_kernel(const half_t* __restrict__ x, const int32_t* __restrict__ index,
                                                           SlotPlan plan, Layers layers, int T, half_t* __restrict__ out) {
  const int p = blockIdx.x;
  if (p >= plan.counts[1]) return;
  const int slot = plan.order[p], K = layers.K;
  const int32_t* at = layers.order(index ? index[slot] : 0);
  const half_t* row = x + static_cast<size_t>(slot / T) * K;
  for (int i = 8 * threadIdx.x; i < K; i += 8 * 256) {
    half8_t v;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = row[min(static_cast<uint32_t>(at[i + j]), static_cast<uint32_t>(K - 1))];
    *reinterpret_cast<half8_t*>(out + static_cast<size_t>(p) * K + i) = v;
  }
}

// Input channel -> stored position of every expert: inverse[e][order(e)[i]] = i.
__global__ __launch_bounds__(256) void invert_order_kernel(Layers layers, int32_t* __restrict__ inverse) {
  const int i = blockIdx.x * 256 + threadIdx.x, e = blockIdx.y, K = layers.K;
  if (i >= K) return;
  const uint32_t k = layers.order(e)[i];
  if (k < static_cast<uint32_t>(K)) inverse[static_cast<size_t>(e) * K + k] = i;
}

}  // namespace w4a16
