// Slots grouped by expert:
//  * each wavefront counts the experts of its own run of slots in an LDS histogram of its
//    own; a scan over the wavefronts of every expert and over the experts gives every
//    wavefront the place of its first slot of every expert;
//  * the second pass ranks the 64 slots of a load among themselves by ballots over the bits
//    of the expert's number (10 at most), so that the order is stable and does not depend on
//    timing.
// Slots without an expert come last, in no tile.  Bound by the latency of the two passes: 8
// loads of 64 slots per wavefront are in flight at once.  Up to kPlanSlots slots one workgroup
// does it all; more are counted by many, scanned by one and placed by many (2^16 slots of 128
// experts 71 us by one workgroup, 17 us by 32; 2^20 slots 1430 us, 40 us by 256).  And the
// channel orders of act order.
#pragma once

#include "plan.hpp"

namespace w4a16 {

// A wavefront's run of slots, [begin, end), of index outside [0, limit): no expert; index NULL:
// expert 0 for every slot.  E == limit, or E == 1: every slot with an index inside belongs to
// expert 0.
struct SlotRun {
  static constexpr int U = 8;   // loads in flight
  const int32_t* index;
  int begin, end, E, limit, lane;

  __device__ __forceinline__ SlotRun(const int32_t* index_, int64_t from, int64_t to, int E_, int limit_, int tid)
      : index(index_), E(E_), limit(limit_), lane(tid & 63) {
    const int64_t run = ((to - from + kPlanWaves - 1) / kPlanWaves + 63) / 64 * 64;
    begin = static_cast<int>(min(to, from + (tid >> 6) * run));
    end = static_cast<int>(min(to, begin + run));
  }
  __device__ __forceinline__ int expert_of(int s) const {
    if (s >= end) return -1;   // no slot
    const int e = index ? index[s] : 0;
    return e < 0 || e >= limit ? E : E == 1 ? 0 : e;
  }
  // f(first slot of 64, this lane's expert or -1), in order
  template <class F>
  __device__ __forceinline__ void each(F f) const {
    for (int s0 = begin; s0 < end; s0 += 64 * U) {
      int e[U];
#pragma unroll
      for (int u = 0; u < U; ++u) e[u] = expert_of(min(s0 + 64 * u, end) + lane);
#pragma unroll
      for (int u = 0; u < U; ++u) f(s0 + 64 * u, e[u]);
    }
  }
  __device__ __forceinline__ void count(int32_t* mine) const {
    each([&](int, int e) {
      if (e >= 0) atomicAdd(&mine[e], 1);
    });
  }
  // mine[e]: slots of expert e before the run.
  __device__ __forceinline__ void place(int32_t* mine, const int32_t* first, const int32_t* tile0, int height,
                                        const SlotPlan& plan) const {
    const int bits = 32 - __clz(E);
    each([&](int s0, int e) {
      unsigned long long same = __ballot(e >= 0);
      for (int b = 0; b < bits; ++b) {
        const unsigned long long set = __ballot((e >> b) & 1);
        same &= (e >> b) & 1 ? set : ~set;
      }
      const int rank = __popcll(same & ((1ull << lane) - 1));
      if (e >= 0) {
        const int within = mine[e] + rank;
        plan.order[first[e] + within] = s0 + lane;
        if (plan.tile_of) plan.tile_of[s0 + lane] = tile0[e] + within / height;
      }
      __builtin_amdgcn_wave_barrier();
      if (e >= 0 && rank == 0) mine[e] += __popcll(same);
      __builtin_amdgcn_wave_barrier();
    });
  }
};

// The counts of the wavefronts, hist [kPlanWaves][E + 1], become the slots before each
// wavefront's run, `before` of them before the first; returns the sum (thread e, expert e).
__device__ __forceinline__ int scan_waves(int32_t* hist, int bins, int e, int before) {
  for (int w = 0; w < kPlanWaves; ++w) {
    const int c = hist[w * bins + e];
    hist[w * bins + e] = before;
    before += c;
  }
  return before;
}

// First place and first tile of every expert, and the tiles, from the experts' counts (thread
// e, expert e; E the slots without one).  All threads; ends with a barrier.
__device__ __forceinline__ void list_tiles(int count, int E, int height, const SlotPlan& plan, int32_t* first, int32_t* tile0) {
  __shared__ int32_t wave_sum[kPlanWaves][2];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int tiles = tid < E ? count / height + (count % height != 0) : 0;
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
  if (tid <= E) first[tid] = pc, tile0[tid] = pt;
  if (tid == E) {
    plan.counts[0] = pt;
    plan.counts[1] = pc;
  }
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
}

__global__ __launch_bounds__(kPlanThreads) void plan_slots_kernel(const int32_t* __restrict__ index, int S, int E,
                                                                  int limit, int height, SlotPlan plan) {
  extern __shared__ int32_t hist[];   // [kPlanWaves][E + 1]
  __shared__ int32_t first[kMaxExperts + 2];
  __shared__ int32_t tile0[kMaxExperts + 2];
  const int tid = threadIdx.x, bins = E + 1;
  for (int i = tid; i < kPlanWaves * bins; i += kPlanThreads) hist[i] = 0;
  __syncthreads();
  const SlotRun run(index, 0, S, E, limit, tid);
  int32_t* mine = hist + (tid >> 6) * bins;
  run.count(mine);
  __syncthreads();
  const int count = tid < bins ? scan_waves(hist, bins, tid, 0) : 0;
  list_tiles(count, E, height, plan, first, tile0);
  run.place(mine, first, tile0, height, plan);
}

// The same in three launches.  sums [blocks + 2][E + 1]: the workgroups' counts, then the slots of
// every expert before each workgroup's, the experts' first places and their first tiles.
__global__ __launch_bounds__(kPlanThreads) void plan_count_kernel(const int32_t* __restrict__ index, int S, int per, int E,
                                                                  int limit, int32_t* __restrict__ sums) {
  extern __shared__ int32_t hist[];   // [E + 1]
  const int tid = threadIdx.x, bins = E + 1;
  for (int i = tid; i < bins; i += kPlanThreads) hist[i] = 0;
  __syncthreads();
  const int64_t from = static_cast<int64_t>(blockIdx.x) * per;
  SlotRun(index, from, min(static_cast<int64_t>(S), from + per), E, limit, tid).count(hist);
  __syncthreads();
  if (tid < bins) sums[static_cast<size_t>(blockIdx.x) * bins + tid] = hist[tid];
}

__global__ __launch_bounds__(kPlanThreads) void plan_scan_kernel(int blocks, int E, int height, SlotPlan plan,
                                                                 int32_t* __restrict__ sums) {
  const int tid = threadIdx.x, bins = E + 1;
  int count = 0;
  if (tid < bins) {
    int32_t* at = sums + tid;
    for (int b0 = 0; b0 < blocks; b0 += 8) {
      int c[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) c[u] = b0 + u < blocks ? at[static_cast<size_t>(b0 + u) * bins] : 0;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (b0 + u < blocks) at[static_cast<size_t>(b0 + u) * bins] = count;
        count += c[u];
      }
    }
  }
  int32_t* heads = sums + static_cast<size_t>(blocks) * bins;
  list_tiles(count, E, height, plan, heads, heads + bins);
}

__global__ __launch_bounds__(kPlanThreads) void plan_place_kernel(const int32_t* __restrict__ index, int S, int per, int E,
                                                                  int limit, int height, int blocks, SlotPlan plan,
                                                                  const int32_t* __restrict__ sums) {
  extern __shared__ int32_t hist[];   // [kPlanWaves][E + 1]
  __shared__ int32_t first[kMaxExperts + 2];
  __shared__ int32_t tile0[kMaxExperts + 2];
  const int tid = threadIdx.x, bins = E + 1;
  for (int i = tid; i < kPlanWaves * bins; i += kPlanThreads) hist[i] = 0;
  if (tid < bins) {
    const int32_t* heads = sums + static_cast<size_t>(blocks) * bins;
    first[tid] = heads[tid];
    tile0[tid] = heads[bins + tid];
  }
  __syncthreads();
  const int64_t from = static_cast<int64_t>(blockIdx.x) * per;
  const SlotRun run(index, from, min(static_cast<int64_t>(S), from + per), E, limit, tid);
  int32_t* mine = hist + (tid >> 6) * bins;
  run.count(mine);
  __syncthreads();
  if (tid < bins) scan_waves(hist, bins, tid, sums[static_cast<size_t>(blockIdx.x) * bins + tid]);
  __syncthreads();
  run.place(mine, first, tile0, height, plan);
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
