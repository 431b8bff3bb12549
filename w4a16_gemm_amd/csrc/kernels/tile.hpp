// The forward tile of the grouped products: BM = 32 MB rows by BN = 64 NB outputs of
// y = x W^^T, by 8 wavefronts (2 along the rows x 4 along the outputs).
//
// K advances in tiles of 64 channels through an LDS ring of three stages (two at 8 bits where
// two workgroups share a compute unit), filled as far ahead as that allows by
// loads straight into LDS (direct.hpp); each wavefront expands the codes of its outputs in
// registers right before its MFMAs, 16x16x32 ones where its blocks are 16 MB rows of 128 or an
// odd number of 16-output blocks, else 32x32x16 ones (twice the work per issue).
//  * Rows lie anywhere in x: the lane offsets of the loads are those of the tile's rows, fixed
//    over the K loop, so the gather costs nothing there.  A row is 8 chunks of 8 channels,
//    chunk j of row r at slot j ^ (r / 2 % 8).
//  * Codes: the 32 (64 at 8 bits) bytes of an output are taken by neighbouring lanes of one
//    load, part p of output n at slot p ^ (n / 8 % 2) (p ^ (n / 4 % 4)), so that the lanes
//    that read a part of 16 outputs at once meet distinct banks.
// A row's result does not depend on the other rows of the tile, or on its place in it.
//
// With half the memory, two workgroups per compute unit, a wavefront has 128 registers: it expands
// one block's weights, multiplies, and goes on to the next, where a tile alone on a compute unit
// expands all first.  Expanded at once they spilled 2 to 17 registers, in the head's kernels up to 12 reloads
// for 64 channels (losses of 803 rows against 16512 outputs, K 4096 165 -> 152 us, 100 against 128000, 8
// bits, K 1536 96 -> 80 us; 32 experts of 64 rows, N and K 4096 181 -> 179 us).
#pragma once

#include "direct.hpp"
#include "gemm.hpp"
#include "plan.hpp"

namespace w4a16 {

// BM: rows that a stage has room for.  256: one workgroup per compute unit; 128: two.
template <int BITS, int BM>
struct TileStage {
  static constexpr uint32_t A = BM * 128;
  static constexpr uint32_t C = 256 * 8 * BITS;
  static constexpr uint32_t S = 2 * 256 * 2;                // [half][output]
  static constexpr uint32_t Z = BITS == 4 ? 256 : 1024;     // the same; whole wavefronts' loads
  static constexpr uint32_t BYTES = A + C + S + Z;
  static constexpr int COUNT = BITS == 8 && BM == 128 ? 2 : 3;   // as many as fit
};

// Behind the ring: four words per row of the tile.
template <int BITS, int BM>
constexpr size_t tile_lds() { return TileStage<BITS, BM>::COUNT * static_cast<size_t>(TileStage<BITS, BM>::BYTES) + 16 * BM; }
static_assert(tile_lds<4, 256>() <= 160 * 1024 && tile_lds<8, 256>() <= 160 * 1024, "fits a compute unit");
static_assert(tile_lds<4, 128>() <= 80 * 1024 && tile_lds<8, 128>() <= 80 * 1024, "two workgroups per compute unit");

template <int NB, int MB, int BITS, int BM>
struct TileLoader {
  using L = TileStage<BITS, BM>;
  static constexpr int APT = MB / 2;     // row loads (16 B) per thread and stage
  static constexpr int CL = BITS / 4;    // code loads
  static constexpr int BN = 64 * NB, PARTS = BITS / 2, KBYTES = 8 * BITS;
  u32x4_t xr, qr;
  const half_t* s_ptr;
  const uint32_t* z_ptr;
  uint32_t ring;   // LDS offset
  int KT, gshift, wave, half, s_pitch, z_pitch;
  uint32_t a_off[APT], b_off[CL];

  // rows source[0 .. rows) (LDS) of x, x_rows in all; outputs from n0 on.
  __device__ __forceinline__ TileLoader(const half_t* x, int x_rows, const Layers& l, unsigned char* smem,
                                        const int32_t* source, int rows, int n0, int tid, int wave_)
      : ring(lds_offset(smem)), KT(l.K / 64), gshift(l.gshift), wave(wave_), s_pitch(l.N) {
    const int lane = tid & 63, N = l.N;
    const uint32_t pitch = static_cast<uint32_t>(l.K) * BITS / 8;
    const int here = min(BN, N - n0);
    xr = direct_rsrc(x, static_cast<uint32_t>(x_rows) * l.K * 2u);
    qr = direct_rsrc(reinterpret_cast<const unsigned char*>(l.qw) + static_cast<size_t>(n0) * pitch,
                     static_cast<uint32_t>(here) * pitch);
#pragma unroll
    for (int i = 0; i < APT; ++i) {
      const int c = (wave * APT + i) * 64 + lane, row = c >> 3, slot = c & 7;
      a_off[i] = (static_cast<uint32_t>(source[min(row, rows - 1)]) * l.K + 8 * (slot ^ ((row >> 1) & 7))) * 2u;
    }
#pragma unroll
    for (int i = 0; i < CL; ++i) {
      const int c = tid + 512 * i, n = c / PARTS, slot = c % PARTS;
      const int part = BITS == 4 ? slot ^ ((n >> 3) & 1) : slot ^ ((n >> 2) & 3);
      b_off[i] = static_cast<uint32_t>(min(n, here - 1)) * pitch + 16u * part;
    }
    // wavefront 0: scales, 8 outputs per lane; wavefront 1: zero points, 8 (16) outputs per lane
    half = wave == 0 || BITS == 4 ? lane >> 5 : (lane >> 4) & 1;
    s_ptr = l.scales + min(n0 + 8 * (lane & 31), N - 8);
    const int zn = BITS == 4 ? min(n0 / 8 + (lane & 31), N / 8 - 1) : min(n0 / 4 + 4 * (lane & 15), N / 4 - 4);
    z_ptr = l.zeros.words + (l.zeros.sym ? 0 : zn);
    z_pitch = l.zeros.sym ? 0 : N / (32 / BITS);
  }

  // Tile t to stage t % COUNT; past the end the last one again.  Scales and zero points come
  // first: waiting for tile t waits for no more than those of tile t + 1.
  __device__ __forceinline__ void load(int t) const {
    const uint32_t stage = ring + (t % L::COUNT) * L::BYTES;
    const int tc = min(t, KT - 1);
    const int g = (tc * 64 + 32 * half) >> gshift;
    const uint32_t scales = stage + L::A + L::C;
    if (wave == 0)
      direct_load<16>(s_ptr + static_cast<size_t>(g) * s_pitch, scales);
    else if (wave == 1)
      direct_load<BITS == 4 ? 4 : 16>(z_ptr + static_cast<size_t>(g) * z_pitch, scales + L::S);
    direct_loads16<APT, 1024>(xr, stage + wave * APT * 1024, a_off, tc * 128);
    direct_loads16<CL, 512 * 16>(qr, stage + L::A + wave * 1024, b_off, tc * KBYTES);
  }
};

// Constants of output `col` of the tile for the 32 channels `half` of a stage.
template <int BITS, int BM>
__device__ __forceinline__ DequantConsts tile_consts(const unsigned char* scales, Zeros zeros, int half, int col) {
  using L = TileStage<BITS, BM>;
  const uint32_t sc = *reinterpret_cast<const uint16_t*>(scales + (half * 256 + col) * 2);
  uint32_t z;
  if constexpr (BITS == 4)
    z = (zeros.word(*reinterpret_cast<const uint32_t*>(scales + L::S + (half * 32 + (col >> 3)) * 4)) >> (4 * (col & 7))) & 0xFu;
  else
    z = zeros.sym ? 128u : *(scales + L::S + half * 256 + col);
  return make_consts(z, __builtin_bit_cast(half_t, static_cast<uint16_t>(sc)));
}

// acc[mb][nb]: 16 x 16 blocks of the wavefront's 16 MB rows and 16 NB outputs.  Lane (r, q) has
// the channels [16 q + 8 s, +8) in MFMA step s.
template <int NB, int MB, int BITS, int BM>
__device__ __forceinline__ void tile_product(const TileLoader<NB, MB, BITS, BM>& ld, Zeros zeros, const unsigned char* smem,
                                             int tid, int wave, float4_t (&acc)[MB][NB]) {
  using L = TileStage<BITS, BM>;
  using Loader = TileLoader<NB, MB, BITS, BM>;
  constexpr int INFLIGHT = (L::COUNT - 2) * (Loader::APT + Loader::CL);   // of the tiles after the next
  const int lane = tid & 63, wm = wave >> 2, wn = wave & 3, lr = lane & 15, lq = lane >> 4;
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = float4_t{0.f, 0.f, 0.f, 0.f};
  const int col = wn * 16 * NB + lr;
  const uint32_t a_lane = (wm * 16 * MB + lr) * 128;
#pragma unroll
  for (int t = 0; t < L::COUNT - 1; ++t) ld.load(t);
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(INFLIGHT) : "memory");   // tile 0
  block_barrier();
  DequantConsts dc[NB];
  const int gmask = (1 << min(ld.gshift, 30)) - 1;
  for (int t = 0; t < ld.KT; ++t) {
    ld.load(t + L::COUNT - 1);
    const unsigned char* st = smem + (t % L::COUNT) * L::BYTES;
    uint32_t cw[NB][BITS / 2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int n = col + 16 * nb;
      if constexpr (BITS == 4) {
        const uint2 v = *reinterpret_cast<const uint2*>(st + L::A + n * 32 + (((lq >> 1) ^ ((n >> 3) & 1)) * 16) + (lq & 1) * 8);
        cw[nb][0] = v.x, cw[nb][1] = v.y;
      } else {
        const uint4 v = *reinterpret_cast<const uint4*>(st + L::A + n * 64 + ((lq ^ ((n >> 2) & 3)) * 16));
        cw[nb][0] = v.x, cw[nb][1] = v.y, cw[nb][2] = v.z, cw[nb][3] = v.w;
      }
    }
    // constants are rebuilt only where the tile starts a new group
    if (((t * 64) & gmask) == 0) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) dc[nb] = tile_consts<BITS, BM>(st + L::A + L::C, zeros, lq >> 1, col + 16 * nb);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      half8_t af[MB], bf[NB];
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
        af[mb] = *reinterpret_cast<const half8_t*>(st + a_lane + 16 * ((2 * lq + s) ^ (lr >> 1)) + 2048 * mb);
      auto expand = [&](int nb) {
        if constexpr (BITS == 4) {
          bf[nb] = dequant_word(cw[nb][s], dc[nb]);
        } else {
          const half4_t lo = dequant_word8(cw[nb][2 * s], dc[nb]), hi = dequant_word8(cw[nb][2 * s + 1], dc[nb]);
          bf[nb] = half8_t{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        }
      };
      auto multiply = [&](int mb, int nb) {
        acc[mb][nb] = __builtin_amdgcn_mfma_f32_16x16x32_f16(af[mb], bf[nb], acc[mb][nb], 0, 0, 0);
      };
      if constexpr (BM == 128) {   // one block's weights at a time
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          expand(nb);
#pragma unroll
          for (int mb = 0; mb < MB; ++mb) multiply(mb, nb);
          __builtin_amdgcn_sched_barrier(0);
        }
      } else {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) expand(nb);
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) multiply(mb, nb);
        __builtin_amdgcn_s_setprio(0);
      }
    }
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(INFLIGHT) : "memory");   // tile t + 1; own reads done
    block_barrier();
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the clamped loads past the last tile
}

// acc[rb][cb]: 32 x 32 blocks.  Lane (h, c) = (lane / 32, lane % 32) has the channels
// [32 h + 8 s, +8) in MFMA step s.
template <int NB, int MB, int BITS, int BM>
__device__ __forceinline__ void tile_product32(const TileLoader<NB, MB, BITS, BM>& ld, Zeros zeros, const unsigned char* smem,
                                               int tid, int wave, f32x16_t (&acc)[MB / 2][NB / 2]) {
  using L = TileStage<BITS, BM>;
  using Loader = TileLoader<NB, MB, BITS, BM>;
  constexpr int INFLIGHT = (L::COUNT - 2) * (Loader::APT + Loader::CL);   // of the tiles after the next
  constexpr int RB = MB / 2, CB = NB / 2;
  const int lane = tid & 63, wm = wave >> 2, wn = wave & 3, lc = lane & 31, lh = lane >> 5;
#pragma unroll
  for (int rb = 0; rb < RB; ++rb)
#pragma unroll
    for (int cb = 0; cb < CB; ++cb)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[rb][cb][r] = 0.f;
  const int col = wn * 16 * NB + lc;
  const uint32_t a_lane = (wm * 16 * MB + lc) * 128;
#pragma unroll
  for (int t = 0; t < L::COUNT - 1; ++t) ld.load(t);
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(INFLIGHT) : "memory");   // tile 0
  block_barrier();
  DequantConsts dc[CB];
  const int gmask = (1 << min(ld.gshift, 30)) - 1;
  for (int t = 0; t < ld.KT; ++t) {
    ld.load(t + L::COUNT - 1);
    const unsigned char* st = smem + (t % L::COUNT) * L::BYTES;
    uint4 cw[CB][BITS / 4];
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
      const int n = col + 32 * cb;
      if constexpr (BITS == 4) {
        cw[cb][0] = *reinterpret_cast<const uint4*>(st + L::A + n * 32 + ((lh ^ ((n >> 3) & 1)) * 16));
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          cw[cb][i] = *reinterpret_cast<const uint4*>(st + L::A + n * 64 + (((2 * lh + i) ^ ((n >> 2) & 3)) * 16));
      }
    }
    if (((t * 64) & gmask) == 0) {
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) dc[cb] = tile_consts<BITS, BM>(st + L::A + L::C, zeros, lh, col + 32 * cb);
    }
    // fragments one step ahead: the reads of step s + 1 are in flight during the MFMAs of s
    half8_t af[2][RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
      af[0][rb] = *reinterpret_cast<const half8_t*>(st + a_lane + 4096 * rb + 16 * ((4 * lh) ^ ((lc >> 1) & 7)));
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s < 3) {
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
          af[(s + 1) & 1][rb] = *reinterpret_cast<const half8_t*>(st + a_lane + 4096 * rb + 16 * ((4 * lh + s + 1) ^ ((lc >> 1) & 7)));
      }
      __builtin_amdgcn_sched_barrier(0);   // keep the reads ahead of this step's MFMAs
      half8_t bf[CB];
      auto expand = [&](int cb) {
        if constexpr (BITS == 4) {
          const uint4 c = cw[cb][0];
          bf[cb] = dequant_word(s == 0 ? c.x : s == 1 ? c.y : s == 2 ? c.z : c.w, dc[cb]);
        } else {
          const uint4 c = cw[cb][s >> 1];
          const half4_t lo = dequant_word8((s & 1) ? c.z : c.x, dc[cb]), hi = dequant_word8((s & 1) ? c.w : c.y, dc[cb]);
          bf[cb] = half8_t{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        }
      };
      auto multiply = [&](int rb, int cb) {
        acc[rb][cb] = __builtin_amdgcn_mfma_f32_32x32x16_f16(af[s & 1][rb], bf[cb], acc[rb][cb], 0, 0, 0);
      };
      if constexpr (BM == 128) {   // one block's weights at a time
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) {
          expand(cb);
#pragma unroll
          for (int rb = 0; rb < RB; ++rb) multiply(rb, cb);
          __builtin_amdgcn_sched_barrier(0);
        }
      } else {
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) expand(cb);
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
          for (int cb = 0; cb < CB; ++cb) multiply(rb, cb);
        __builtin_amdgcn_s_setprio(0);
      }
    }
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(INFLIGHT) : "memory");   // tile t + 1; own reads done
    block_barrier();
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the clamped loads past the last tile
}

}  // namespace w4a16
