// Routing of rows to experts, and the weighted sum of their outputs.
//
// Routing: a group of LANES lanes has a row of up to 8 LANES logits in registers.  A logit
// and its index make one 64-bit key that orders by value, then by the lower index; each of
// the top_k rounds takes the largest key of the row (a maximum over the lane's keys, then
// over the lanes) and removes it.  -infinity and NaN have the key 0 and are never taken.
// Softmax statistics are fp32, over all experts.
// The sums are streams: every value of y, dout and dy passes once, 16 bytes per lane.
#pragma once

#include "plan.hpp"

namespace w4a16 {

__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(half_t v) { return static_cast<float>(v); }

__device__ __forceinline__ unsigned long long route_key(float v, int j) {
  const float z = v + 0.f;   // -0 and 0 are equal
  if (!(z > -INFINITY)) return 0;
  const uint32_t b = __builtin_bit_cast(uint32_t, z);
  const uint32_t u = b ^ (b >> 31 ? 0xFFFFFFFFu : 0x80000000u);
  return static_cast<unsigned long long>(u) << 32 | static_cast<uint32_t>(~j);
}
__device__ __forceinline__ float key_value(unsigned long long key) {
  const uint32_t u = static_cast<uint32_t>(key >> 32);
  return __builtin_bit_cast(float, u ^ (u >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}

template <int CTRL>
__device__ __forceinline__ unsigned long long dpp_key(unsigned long long v) {
  const int lo = __builtin_amdgcn_mov_dpp(static_cast<int>(static_cast<uint32_t>(v)), CTRL, 0xF, 0xF, true);
  const int hi = __builtin_amdgcn_mov_dpp(static_cast<int>(v >> 32), CTRL, 0xF, 0xF, true);
  return static_cast<unsigned long long>(static_cast<uint32_t>(hi)) << 32 | static_cast<uint32_t>(lo);
}
__device__ __forceinline__ unsigned long long larger(unsigned long long a, unsigned long long b) { return a > b ? a : b; }

// Maximum / sum over a group of 16 or 64 neighbouring lanes, in every lane.
template <int LANES>
__device__ __forceinline__ unsigned long long lanes_max(unsigned long long v) {
  static_assert(LANES == 16 || LANES == 64, "16 or 64 lanes");
  v = larger(v, dpp_key<0xB1>(v));    // quad_perm [1, 0, 3, 2]
  v = larger(v, dpp_key<0x4E>(v));    // quad_perm [2, 3, 0, 1]
  v = larger(v, dpp_key<0x141>(v));   // row_half_mirror
  v = larger(v, dpp_key<0x140>(v));   // row_mirror
  if constexpr (LANES == 64) {
    v = larger(v, __shfl_xor(v, 16));
    v = larger(v, __shfl_xor(v, 32));
  }
  return v;
}
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int d = 1; d < LANES; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

// Lane l of a row's group holds the logits l + LANES j, j < PER, and the results of the
// rounds t with t % LANES == l.
template <int LANES, int PER, typename T>
__global__ __launch_bounds__(256) void route_kernel(const T* __restrict__ logits, int M, int E, int top_k, int renorm,
                                                    int32_t* __restrict__ index, float* __restrict__ weights) {
  const int m = blockIdx.x * (256 / LANES) + threadIdx.x / LANES, l = threadIdx.x % LANES;
  const size_t at = static_cast<size_t>(min(m, M - 1));
  const T* row = logits + at * E;
  float v[PER];
  unsigned long long key[PER];
  unsigned long long best = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = l + LANES * j;
    v[j] = e < E ? as_float(row[e]) : -INFINITY;
  }
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    key[j] = route_key(v[j], l + LANES * j);
    best = larger(best, key[j]);
  }
  best = lanes_max<LANES>(best);
  const float top = best ? key_value(best) : 0.f;
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < PER; ++j) sum += expf(v[j] - top);
  const float scale = 1.f / lanes_sum<LANES>(sum);
  float chosen = 0.f;   // sum of this lane's weights
  for (int t0 = 0; t0 < top_k; t0 += LANES) {
    const int rounds = min(LANES, top_k - t0);
    unsigned long long mine = 0;
    for (int t = 0; t < rounds; ++t) {
      if (l == t) mine = best;
      unsigned long long next = 0;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        if (key[j] == best) key[j] = 0;
        next = larger(next, key[j]);
      }
      best = lanes_max<LANES>(next);
    }
    const float w = mine ? expf(key_value(mine) - top) * scale : 0.f;
    chosen += w;
    // renormalised weights of one group of rounds wait for the sum, of several are written
    // and scaled below
    if (l < rounds && m < M) {
      index[at * top_k + t0 + l] = mine ? static_cast<int32_t>(~static_cast<uint32_t>(mine)) : -1;
      if (!renorm || top_k > LANES) weights[at * top_k + t0 + l] = w;
    }
    if (renorm && top_k <= LANES) {
      const float total = lanes_sum<LANES>(chosen);
      if (l < rounds && m < M) weights[at * top_k + l] = mine ? w / total : 0.f;
    }
  }
  if (renorm && top_k > LANES) {
    const float total = lanes_sum<LANES>(chosen);
    for (int t = l; t < top_k && m < M; t += LANES) {   // this lane's own
      const float w = weights[at * top_k + t];
      if (index[at * top_k + t] >= 0) weights[at * top_k + t] = w / total;
    }
  }
}

// Gradient of the logits for that of the weights.  Renormalised weights are a softmax over
// the chosen logits alone: dl = w (dw - sum w dw).  Otherwise w = p: dl_j = [chosen] w dw -
// p_j sum w dw.  Slots with an index outside [0, E) take no part.
template <int LANES, int PER, typename T>
__global__ __launch_bounds__(256) void route_backward_kernel(const float* __restrict__ dweights,
                                                             const T* __restrict__ logits,
                                                             const int32_t* __restrict__ index,
                                                             const float* __restrict__ weights, int M, int E, int top_k,
                                                             int renorm, T* __restrict__ dlogits) {
  const int m = blockIdx.x * (256 / LANES) + threadIdx.x / LANES, l = threadIdx.x % LANES;
  const size_t at = static_cast<size_t>(min(m, M - 1));
  float g[PER];
  if (!renorm) {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int e = l + LANES * j;
      g[j] = e < E ? as_float(logits[at * E + e]) : -INFINITY;
    }
  }
  // a lane's slot: expert, w dw and w (0 where there is none); the last group of slots stays in
  // registers for the second walk
  int e = -1;
  float w = 0.f, wdw = 0.f, part = 0.f;
  auto load = [&](int t) {
    e = t < top_k ? index[at * top_k + t] : -1;
    const bool valid = e >= 0 && e < E;
    if (!valid) e = -1;
    w = valid ? weights[at * top_k + t] : 0.f;
    wdw = valid ? w * dweights[at * top_k + t] : 0.f;
  };
  for (int t0 = 0; t0 < top_k; t0 += LANES) {
    load(t0 + l);
    part += wdw;
  }
  const float mean = lanes_sum<LANES>(part);
  if (renorm) {
#pragma unroll
    for (int j = 0; j < PER; ++j) g[j] = 0.f;
  } else {
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < PER; ++j) top = fmaxf(top, g[j]);
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    if (top == -INFINITY) top = 0.f;
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      g[j] = expf(g[j] - top);
      sum += g[j];
    }
    sum = lanes_sum<LANES>(sum);
    const float scale = sum == 0.f ? 0.f : -mean / sum;   // no expert has a finite logit: no gradient
#pragma unroll
    for (int j = 0; j < PER; ++j) g[j] *= scale;
  }
  for (int t0 = 0; t0 < top_k; t0 += LANES) {
    if (top_k > LANES) load(t0 + l);
    const float d = renorm ? wdw - w * mean : wdw;
    const int rounds = min(LANES, top_k - t0);
    for (int t = 0; t < rounds; ++t) {
      const int from = (threadIdx.x & 63 & ~(LANES - 1)) + t;
      const int et = __shfl(e, from);
      const float dt = __shfl(d, from);
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (et == l + LANES * j) g[j] += dt;
    }
  }
  if (m >= M) return;
#pragma unroll
  for (int j = 0; j < PER; ++j)
    if (l + LANES * j < E) dlogits[at * E + l + LANES * j] = static_cast<T>(g[j]);
}

// out[m] = sum_t weights[m][t] y[m][t], fp32, rounded once.  Eight outputs per thread.
__global__ __launch_bounds__(256) void combine_kernel(const half_t* __restrict__ y, const float* __restrict__ weights,
                                                      int64_t runs, int T, int N, half_t* __restrict__ out) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= runs) return;
  const int64_t m = i / (N / 8);
  const int n = static_cast<int>(i % (N / 8)) * 8;
  const half_t* row = y + m * T * N + n;
  float s[8] = {};
#pragma unroll 4
  for (int t = 0; t < T; ++t) {
    const half8_t v = *reinterpret_cast<const half8_t*>(row + static_cast<int64_t>(t) * N);
    const float w = weights[m * T + t];
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] += w * static_cast<float>(v[j]);
  }
  half8_t o;
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = static_cast<half_t>(s[j]);
  *reinterpret_cast<half8_t*>(out + m * N + n) = o;
}

// dy[m][t] = weights[m][t] dout[m], dweights[m][t] = <dout[m], y[m][t]>: one workgroup per
// row, four slots at a time, sums in a fixed order.
constexpr int kCombineSlots = 4;
__global__ __launch_bounds__(256) void combine_backward_kernel(const half_t* __restrict__ dout,
                                                               const half_t* __restrict__ y,
                                                               const float* __restrict__ weights, int T, int N,
                                                               half_t* __restrict__ dy, float* __restrict__ dweights) {
  __shared__ float red[4][kCombineSlots];
  const int64_t m = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int t0 = 0; t0 < T; t0 += kCombineSlots) {
    float w[kCombineSlots], s[kCombineSlots];
#pragma unroll
    for (int u = 0; u < kCombineSlots; ++u) {
      w[u] = weights[m * T + min(t0 + u, T - 1)];
      s[u] = 0.f;
    }
    for (int n = 8 * threadIdx.x; n < N; n += 8 * 256) {
      const half8_t d = *reinterpret_cast<const half8_t*>(dout + m * N + n);
#pragma unroll
      for (int u = 0; u < kCombineSlots; ++u) {
        if (t0 + u >= T) break;
        const int64_t at = (m * T + t0 + u) * N + n;
        const half8_t v = *reinterpret_cast<const half8_t*>(y + at);
        half8_t o;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          s[u] += static_cast<float>(d[j]) * static_cast<float>(v[j]);
          o[j] = static_cast<half_t>(w[u] * static_cast<float>(d[j]));
        }
        *reinterpret_cast<half8_t*>(dy + at) = o;
      }
    }
#pragma unroll
    for (int u = 0; u < kCombineSlots; ++u) {
      s[u] = lanes_sum<64>(s[u]);
      if (lane == 0) red[wave][u] = s[u];
    }
    __syncthreads();
    if (threadIdx.x < kCombineSlots && t0 + threadIdx.x < T)
      dweights[m * T + t0 + threadIdx.x] =
          (red[0][threadIdx.x] + red[1][threadIdx.x]) + (red[2][threadIdx.x] + red[3][threadIdx.x]);
    __syncthreads();
  }
}

}  // namespace w4a16
