// Tiles of up to 64 rows by 256 outputs: y = x W^^T where the weights' stream bounds the
// product (64 rows are 128 operations per byte of 4-bit codes, below what the matrix cores
// and the memory balance at).
//  * The 8 wavefronts share the rows and split the outputs, 32 each, so that every weight is
//    expanded once (in the tile of gemm.hpp two wavefronts expand the same columns), on
//    32x32x16 MFMAs: lane (h, c) = (lane / 32, lane % 32) has channels [32 h + 8 s, +8) of
//    output c in step s, as in the 32x32 tile there.
//  * K advances in tiles of 64 channels through an LDS ring of low_stages() small stages: rows
//    8 KB, codes 8 KB (16 KB at 8 bits), scales and zero points; two workgroups fit a compute
//    unit, so one's start and end hide behind the other's loop.
//  * Tile t is waited for and a barrier passed before tile t + stages - 1 is requested into the
//    stage of tile t - 1, which every wavefront has left by then.
// Measured, 37 rows against a head of 151936 outputs, K 1536: 112 us -> KEPT us in this tile.
#pragma once

#include "experts.hpp"

namespace w4a16 {

template <int BITS>
struct LowStage {
  static constexpr uint32_t A = 64 * 64 * 2;
  static constexpr uint32_t C = 256 * 64 * BITS / 8;
  static constexpr uint32_t S = 2 * 256 * 2;                    // [half][output]
  static constexpr uint32_t Z = BITS == 4 ? 256 : 1024;         // [half][output], 64 lanes' loads
  static constexpr uint32_t BYTES = A + C + S + Z;
  static constexpr int COUNT = BITS == 4 ? 4 : 3;               // two workgroups' rings in 160 KB
};

constexpr size_t kLowRowsLds = 4 * 64 * 4;   // four words per row, behind the ring

template <int BITS>
constexpr size_t low_lds() { return static_cast<size_t>(LowStage<BITS>::COUNT) * LowStage<BITS>::BYTES + kLowRowsLds; }
static_assert(low_lds<4>() <= 80 * 1024 && low_lds<8>() <= 80 * 1024, "two workgroups per compute unit");

template <int BITS>
struct LowLoader {
  using L = LowStage<BITS>;
  static constexpr int CL = BITS / 4;   // code loads per thread and stage
  __amdgpu_buffer_rsrc_t xr, qr;
  const half_t* s_ptr;
  const uint32_t* z_ptr;
  Zeros zeros;
  unsigned char* smem;
  int N, KT, gshift, wave, half;
  uint32_t a_off, b_off[CL];

  __device__ __forceinline__ LowLoader(const half_t* x, int x_rows, const Layers& l, unsigned char* smem_,
                                       const int32_t* source, int rows, int n0, int tid, int wave_)
      : zeros(l.zeros), smem(smem_), N(l.N), KT(l.K / 64), gshift(l.gshift), wave(wave_) {
    const int lane = tid & 63;
    const uint32_t pitch = static_cast<uint32_t>(l.K) * BITS / 8;
    xr = __builtin_amdgcn_make_buffer_rsrc(const_cast<half_t*>(x), 0,
                                           static_cast<int>(static_cast<uint32_t>(x_rows) * l.K * 2u), kBufferWord3);
    qr = __builtin_amdgcn_make_buffer_rsrc(
        reinterpret_cast<unsigned char*>(const_cast<uint32_t*>(l.qw)) + static_cast<size_t>(n0) * pitch, 0,
        static_cast<int>(static_cast<uint32_t>(min(256, l.N - n0)) * pitch), kBufferWord3);
    // rows: chunk tid = 8 row + slot receives the row's chunk slot ^ (row % 8)
    const int row = tid >> 3, slot = tid & 7;
    a_off = (static_cast<uint32_t>(source[min(row, rows - 1)]) * l.K + 8 * (slot ^ (row & 7))) * 2u;
    // codes: chunk c = part * 256 + output holds the part's channels (32 at 4 bits, 16 at 8)
#pragma unroll
    for (int i = 0; i < CL; ++i) {
      const int c = tid + 512 * i;
      b_off[i] = static_cast<uint32_t>(min(c % 256, l.N - 1 - n0)) * pitch + 16u * (c / 256);
    }
    half = lane >> 5;
    s_ptr = l.scales + min(n0 + 8 * (lane & 31), N - 8);
    const int n = BITS == 4 ? min(n0 / 8 + (lane & 31), N / 8 - 1) : min(n0 / 4 + 4 * (lane & 31), N / 4 - 4);
    z_ptr = l.zeros.words + (l.zeros.sym ? 0 : n);
  }

  // Tile t to stage t % COUNT; past the end the last one again.
  __device__ __forceinline__ void load(int t) const {
    unsigned char* stage = smem + (t % L::COUNT) * L::BYTES;
    const int tc = min(t, KT - 1);
    const int g = (tc * 64 + 32 * half) >> gshift;
    if (wave == 0)
      __builtin_amdgcn_global_load_lds(reinterpret_cast<const void*>(s_ptr + static_cast<size_t>(g) * N),
                                       reinterpret_cast<void*>(stage + L::A + L::C), 16, 0, 0);
    else if (wave == 1) {
      const uint32_t* z = z_ptr + (zeros.sym ? 0 : static_cast<size_t>(g) * (N / (32 / BITS)));
      if constexpr (BITS == 4)
        __builtin_amdgcn_global_load_lds(reinterpret_cast<const void*>(z),
                                         reinterpret_cast<void*>(stage + L::A + L::C + L::S), 4, 0, 0);
      else
        __builtin_amdgcn_global_load_lds(reinterpret_cast<const void*>(z),
                                         reinterpret_cast<void*>(stage + L::A + L::C + L::S), 16, 0, 0);
    }
    __builtin_amdgcn_raw_ptr_buffer_load_lds(xr, as_lds(stage + wave * 1024), 16, static_cast<int>(a_off), tc * 128, 0, 0);
    unsigned char* codes = stage + L::A;
#pragma unroll
    for (int i = 0; i < CL; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(qr, as_lds(codes + (512 * i + wave * 64) * 16), 16,
                                               static_cast<int>(b_off[i]), tc * (8 * BITS), 0, 0);
  }

  // Waits for this wavefront's loads of all but the newest COUNT - 2 tiles.
  __device__ __forceinline__ void wait() const {
    if (wave < 2)
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"((L::COUNT - 2) * (CL + 2)) : "memory");
    else
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"((L::COUNT - 2) * (CL + 1)) : "memory");
  }
};

template <int RB>
struct LowSums {
  f32x16_t b[RB];
};

// acc.b[i]: rows 32 i .. of the tile, outputs 32 wave .. +32 (D layout of the 32x32 MFMA).
// RB: 32-row blocks (rows past 32 RB are not computed).
template <int BITS, int RB>
__device__ __forceinline__ void low_product(const LowLoader<BITS>& ld, Zeros zeros, unsigned char* smem, int tid, int wave,
                                            LowSums<RB>& acc) {
  using L = LowStage<BITS>;
  const int lane = tid & 63, lc = lane & 31, lh = lane >> 5;
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc.b[b][r] = 0.f;
  const int col = wave * 32 + lc;
  const uint32_t a_lane = lc * 128;
  const uint32_t c_lane = L::A + ((BITS == 4 ? lh : 2 * lh) * 256 + col) * 16;
  const uint32_t s_lane = L::A + L::C + (lh * 256 + col) * 2;
  const uint32_t z_lane = L::A + L::C + L::S + (BITS == 4 ? (lh * 32 + (col >> 3)) * 4 : lh * 512 + col);
#pragma unroll
  for (int t = 0; t < L::COUNT - 1; ++t) ld.load(t);
  DequantConsts dc;
  const int gmask = (1 << min(ld.gshift, 30)) - 1;
  for (int t = 0; t < ld.KT; ++t) {
    ld.wait();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    block_barrier();
    ld.load(t + L::COUNT - 1);
    const unsigned char* st = smem + (t % L::COUNT) * L::BYTES;
    uint4 cw[BITS / 4];
    cw[0] = *reinterpret_cast<const uint4*>(st + c_lane);
    if constexpr (BITS == 8) cw[1] = *reinterpret_cast<const uint4*>(st + c_lane + 4096);
    if (((t * 64) & gmask) == 0) {
      const uint32_t sc = *reinterpret_cast<const uint16_t*>(st + s_lane);
      uint32_t z;
      if constexpr (BITS == 4)
        z = (zeros.word(*reinterpret_cast<const uint32_t*>(st + z_lane)) >> (4 * (lc & 7))) & 0xFu;
      else
        z = zeros.sym ? 128u : *(st + z_lane);
      dc = make_consts(z, __builtin_bit_cast(half_t, static_cast<uint16_t>(sc)));
    }
    half8_t af[2][RB];
#pragma unroll
    for (int b = 0; b < RB; ++b)
      af[0][b] = *reinterpret_cast<const half8_t*>(st + a_lane + 4096 * b + 16 * ((4 * lh) ^ (lc & 7)));
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s < 3) {
#pragma unroll
        for (int b = 0; b < RB; ++b)
          af[(s + 1) & 1][b] = *reinterpret_cast<const half8_t*>(st + a_lane + 4096 * b + 16 * ((4 * lh + s + 1) ^ (lc & 7)));
      }
      __builtin_amdgcn_sched_barrier(0);   // keep the reads ahead of this step's MFMAs
      half8_t w;
      if constexpr (BITS == 4) {
        w = dequant_word(s == 0 ? cw[0].x : s == 1 ? cw[0].y : s == 2 ? cw[0].z : cw[0].w, dc);
      } else {
        const uint4 q = cw[s >> 1];
        const half4_t lo = dequant_word8((s & 1) ? q.z : q.x, dc), hi = dequant_word8((s & 1) ? q.w : q.y, dc);
        w = half8_t{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      }
#pragma unroll
      for (int b = 0; b < RB; ++b) acc.b[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(af[s & 1][b], w, acc.b[b], 0, 0, 0);
    }
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");   // the clamped loads past the last tile
}

// Rows of 32 outputs of a wavefront as runs of 8, turned in LDS as in store_tile.
template <int RB, class Value, class Put>
__device__ __forceinline__ void store_low(const LowSums<RB>& acc, unsigned char* smem, int tid, Value value, Put put) {
  constexpr int PITCH = 40;
  const int lane = tid & 63, wave = tid >> 6, lc = lane & 31, lh = lane >> 5;
  half_t* turn = reinterpret_cast<half_t*>(smem) + wave * 32 * PITCH;
#pragma unroll
  for (int b = 0; b < RB; ++b) {
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int row = 8 * (r >> 2) + 4 * lh + (r & 3);
      turn[row * PITCH + lc] = value(32 * b + row, 32 * wave + lc, acc.b[b][r]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = i * 64 + lane, row = at >> 2, run = at & 3;
      put(32 * b + row, 32 * wave + 8 * run, *reinterpret_cast<const half8_t*>(turn + row * PITCH + 8 * run));
    }
  }
}

template <int RB, int BITS>
__device__ __forceinline__ void low_tile(const half_t* x, int x_rows, const Layers& l, half_t* y, unsigned char* smem,
                                         const int32_t* source, const int32_t* slots, int rows, int n0) {
  const int tid = threadIdx.x, N = l.N;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const LowLoader<BITS> ld(x, x_rows, l, smem, source, rows, n0, tid, wave);
  LowSums<RB> acc;
  low_product(ld, l.zeros, smem, tid, wave, acc);
  __syncthreads();
  store_low<RB>(
      acc, smem, tid, [&](int, int, float v) { return static_cast<half_t>(v); },
      [&](int row, int col, half8_t v) {
        if (row < rows && n0 + col < N) *reinterpret_cast<half8_t*>(y + static_cast<size_t>(slots[row]) * N + n0 + col) = v;
      });
}

// experts_gemm_kernel for plans of 64-row tiles.
template <int BITS>
__global__ __launch_bounds__(512, 4) void experts_low_kernel(const half_t* __restrict__ x, int x_rows, int gathered, int T,
                                                             Layers layers, SlotPlan plan, half_t* __restrict__ y) {
  extern __shared__ __align__(16) unsigned char smem[];
  const int tid = threadIdx.x, N = layers.N;
  RowTile tile;
  int col;
  if (!find_tile(plan, (N + 255) / 256, blockIdx.x, tile, col)) return;
  int32_t* slots = reinterpret_cast<int32_t*>(smem + low_lds<BITS>() - kLowRowsLds);
  int32_t* source = slots + 64;
  if (tid < tile.rows) {
    const int s = plan.order[tile.first + tid];
    slots[tid] = s;
    source[tid] = gathered ? tile.first + tid : s / T;
  }
  __syncthreads();
  const int n0 = col * 256;
  if (tile.expert < 0) {   // slots without an expert
    const int cols = min(256, N - n0);
    for (int i = tid; i < tile.rows * (cols / 8); i += 512)
      *reinterpret_cast<half8_t*>(y + static_cast<size_t>(slots[i / (cols / 8)]) * N + n0 + i % (cols / 8) * 8) = half8_t{};
    return;
  }
  const Layers l = layers.at<BITS>(tile.expert);
  if (tile.rows > 32)
    low_tile<2, BITS>(x, x_rows, l, y, smem, source, slots, tile.rows, n0);
  else
    low_tile<1, BITS>(x, x_rows, l, y, smem, source, slots, tile.rows, n0);
}

}  // namespace w4a16
