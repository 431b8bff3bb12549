// Activation checkpoints in 8 bits: the layer's input kept for the backward pass as one
// byte per value and one binary16 scale per row and group of 32 / 64 / 128 channels (the
// int8 absmax scheme of "LLM Quantization: INT8, GPTQ, and AWQ Explained", What
// quantization actually does, applied to activations).
//
//   a = max |x|,  S = smallest binary16 >= a / 127  (1 if a == 0, at most 515.5)
//   q = clamp(round(x / S), -127, 127),  code = q + 128,  value = binary16(q S)
//
// Exactness in fp32.  a / 127 rounded to fp32 and then to binary16 gives a neighbour of
// the true quotient, and 127 h is exact in fp32 (11 + 7 bits), so one comparison with a
// decides whether the next binary16 is needed.  x / S is a quotient of two 11-bit
// significands: unless it is exactly halfway between two integers it is at least 2^-12 away
// from that for |q| <= 128.  It is computed as t = x r with r = fl(1 / S) and one correction t
// + (x - t S) r: the residual is a few ulps of t times S, exact in fp32, so the result is
// within an ulp (2^-17) of the quotient, and equal to it where it is representable, as the
// halfway values are; rint of it is the rounded true quotient.  (A division per value cost
// more than the memory traffic: 8192 x 8192 values 57 us with it, 39 us without.)
// 515.5 is the largest binary16 whose 127-fold still rounds to a finite binary16; a group
// above it (a in {65472, 65504}) has x / S < 127.5 and keeps q = 127.
#pragma once

#include "nibbles.hpp"

namespace w4a16 {

constexpr float kActMaxScale = 515.5f;

// S of a group with largest magnitude a (not NaN, finite).
__device__ __forceinline__ half_t act_scale(float a) {
  half_t h = static_cast<half_t>(a / 127.0f);
  if (static_cast<float>(h) * 127.0f < a)
    h = __builtin_bit_cast(half_t, static_cast<uint16_t>(__builtin_bit_cast(uint16_t, h) + 1));
  if (static_cast<float>(h) > kActMaxScale) h = static_cast<half_t>(kActMaxScale);
  return a == 0.0f ? static_cast<half_t>(1.0f) : h;
}

// One lane quantises 2 x 8 consecutive channels (16 bytes in, 8 bytes out each); a group is
// LPG = group / 8 neighbouring lanes, whose maximum is formed with lane exchanges.
// HBM-bound: 3 bytes per value, 5.2 TB/s at 8192 x 8192.  The codes are written past the L2,
// their reader being the backward pass.  A NaN or an infinity in a group makes its scale
// NaN (codes 128), so that the restored values are NaN and the gradients show it.
constexpr int kActRuns = 2;   // of 256 lanes per workgroup

template <int LPG>
__global__ __launch_bounds__(256) void act_quantize_kernel(const half_t* __restrict__ x, uint8_t* __restrict__ codes,
                                                           half_t* __restrict__ scales, size_t chunks) {
  const size_t first = static_cast<size_t>(blockIdx.x) * 256 * kActRuns + threadIdx.x;
  half8_t v[kActRuns];
#pragma unroll
  for (int k = 0; k < kActRuns; ++k) {
    const size_t i = first + 256 * k;
    v[k] = i < chunks ? reinterpret_cast<const half8_t*>(x)[i] : half8_t{};   // whole groups: LPG divides chunks
  }
#pragma unroll
  for (int k = 0; k < kActRuns; ++k) {
    const size_t i = first + 256 * k;
    float a = 0.0f;
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float f = __builtin_fabsf(static_cast<float>(v[k][e]));
      bad |= !(f <= 65504.0f);
      a = f > a ? f : a;
    }
    if (bad) a = __builtin_inff();
#pragma unroll
    for (int d = 1; d < LPG; d <<= 1) a = fmaxf(a, __shfl_xor(a, d));
    if (i >= chunks) continue;
    const bool finite = a <= 65504.0f;
    const half_t s = finite ? act_scale(a) : __builtin_bit_cast(half_t, static_cast<uint16_t>(0x7E00));
    const float sf = static_cast<float>(s), r = 1.0f / sf;
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float xv = static_cast<float>(v[k][e]);
      const float t = xv * r;
      const float q = fminf(fmaxf(rintf(fmaf(fmaf(-t, sf, xv), r, t)), -127.0f), 127.0f);
      const uint32_t c = finite ? static_cast<uint32_t>(static_cast<int>(q) + 128) : 128u;
      w[e >> 2] |= c << (8 * (e & 3));
    }
    typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
    __builtin_nontemporal_store(u32x2_t{w[0], w[1]}, reinterpret_cast<u32x2_t*>(codes) + i);
    if (i % LPG == 0) scales[i / LPG] = s;
  }
}

// binary16(q S) for two codes placed in the low bytes of the two halves of `pair`: 0x6400
// | c is binary16 1024 + c exactly, minus 1152 is q = c - 128 exactly, so the product is
// the only rounding.
__device__ __forceinline__ uint32_t act_value_pair(uint32_t pair, half2_t s) {
  const half2_t q = as_h2(pair | kMagic) + half2_t{static_cast<half_t>(-1152.0f), static_cast<half_t>(-1152.0f)};
  return __builtin_bit_cast(uint32_t, q * s);
}

// Values of 8 consecutive codes of one group.
__device__ __forceinline__ half8_t act_values(uint2 c, half2_t s) {
  return __builtin_bit_cast(half8_t, (u32x4_t{act_value_pair(__builtin_amdgcn_perm(0u, c.x, 0x0C010C00u), s),
                                              act_value_pair(__builtin_amdgcn_perm(0u, c.x, 0x0C030C02u), s),
                                              act_value_pair(__builtin_amdgcn_perm(0u, c.y, 0x0C010C00u), s),
                                              act_value_pair(__builtin_amdgcn_perm(0u, c.y, 0x0C030C02u), s)}));
}

// Restores 8 consecutive values per lane.  HBM-bound: 8192 x 8192 in 34 us, 5.9 TB/s.
__global__ __launch_bounds__(256) void act_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                             const half_t* __restrict__ scales,
                                                             half_t* __restrict__ x, size_t chunks, int lpg_shift) {
  const size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= chunks) return;
  const uint2 c = reinterpret_cast<const uint2*>(codes)[i];
  const half_t s = scales[i >> lpg_shift];
  reinterpret_cast<half8_t*>(x)[i] = act_values(c, half2_t{s, s});
}

}  // namespace w4a16
