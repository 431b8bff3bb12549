// Tiles of up to 64 rows by 256 outputs: y = x W^^T where the weights' stream bounds the
// product (64 rows are 256 operations per byte of 4-bit codes, below what the matrix cores
// and the memory balance at).
//  * The 8 wavefronts share the rows and split the outputs, 32 each, so that every weight is
//    expanded once (in tile.hpp two wavefronts expand the same columns), on
//    32x32x16 MFMAs: lane (h, c) = (lane / 32, lane % 32) has the 8 channels 64 v + 32 h +
//    8 s of output c in step s of the v-th 64 channels of a stage.
//  * K advances through an LDS ring in stages of 64 bytes of codes per output (128 channels
//    at 4 bits, 64 at 8), so that four neighbouring lanes of a load take one whole piece of a
//    row: stages of 64 channels, 32 bytes per row, were bound by the cache lines that a load
//    touches and by the work per stage (37 rows against a head of 151936 outputs, K 1536: 80
//    us against 66 us).  Two workgroups fit a compute unit, so one's start, end and waits
//    hide behind the other's work.
//  * Stage t is waited for and a barrier passed before stage t + COUNT - 1 is requested into
//    the memory of stage t - 1, which every wavefront has left by then.
//  * Rows: 16 bytes of 8 channels are a chunk; chunk j of row r lies at slot j ^ (r % 16) (8
//    at 64 channels).  Codes: 16-byte part p of output n lies at slot p ^ (n / 4 % 4) of its
//    four.  So 16 lanes that read one chunk of 16 rows, or one part of 16 outputs, meet
//    distinct banks.
#pragma once

#include "experts.hpp"

namespace w4a16 {

template <int BITS>
struct LowStage {
  static constexpr int BK = 512 / BITS;                         // channels
  static constexpr int HALVES = BK / 32;                        // 32-channel parts with a group each
  static constexpr uint32_t ROW = BK * 2;
  static constexpr uint32_t A = 64 * ROW;
  static constexpr uint32_t C = 256 * 64;
  static constexpr uint32_t S = HALVES * 256 * 2;               // [32 channels][output]
  static constexpr uint32_t Z = BITS == 4 ? 512 : 1024;         // the same; whole wavefronts' loads
  static constexpr uint32_t BYTES = A + C + S + Z;
  static constexpr int COUNT = BITS == 4 ? 2 : 3;               // two workgroups' rings in 160 KB
};

constexpr size_t kLowRowsLds = 4 * 64 * 4;   // four words per row, behind the ring

template <int BITS>
constexpr size_t low_lds() { return static_cast<size_t>(LowStage<BITS>::COUNT) * LowStage<BITS>::BYTES + kLowRowsLds; }
static_assert(low_lds<4>() <= 80 * 1024 && low_lds<8>() <= 80 * 1024, "two workgroups per compute unit");

template <int BITS>
struct LowLoader {
  using L = LowStage<BITS>;
  static constexpr int BK = L::BK;
  static constexpr int CPR = BK / 8;               // 16-byte chunks per row
  static constexpr int AL = 64 * CPR / 512;        // row loads per thread and stage
  static constexpr int SW = L::S / 1024;           // wavefronts that load scales, and then zero points
  u32x4_t xr, qr;
  const half_t* s_ptr;
  const uint32_t* z_ptr;
  uint32_t ring;   // LDS offset
  int K, KT, gshift, wave, part, s_pitch, z_pitch;
  uint32_t a_off[AL], b_off[2];

  __device__ __forceinline__ LowLoader(const half_t* x, int x_rows, const Layers& l, unsigned char* smem_,
                                       const int32_t* source, int rows, int n0, int tid, int wave_)
      : ring(lds_offset(smem_)), K(l.K), KT((l.K + L::BK - 1) / L::BK), gshift(l.gshift), wave(wave_), s_pitch(l.N) {
    const int lane = tid & 63, N = l.N;
    const uint32_t pitch = static_cast<uint32_t>(l.K) * BITS / 8;
    xr = direct_rsrc(x, static_cast<uint32_t>(x_rows) * l.K * 2u);
    qr = direct_rsrc(reinterpret_cast<const unsigned char*>(l.qw) + static_cast<size_t>(n0) * pitch,
                     static_cast<uint32_t>(min(256, N - n0)) * pitch);
#pragma unroll
    for (int i = 0; i < AL; ++i) {
      const int c = tid + 512 * i, row = c / CPR, slot = c % CPR;
      a_off[i] = (static_cast<uint32_t>(source[min(row, rows - 1)]) * l.K + 8 * (slot ^ (row & (CPR - 1)))) * 2u;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = tid + 512 * i, n = c >> 2, slot = c & 3;
      b_off[i] = static_cast<uint32_t>(min(n, N - 1 - n0)) * pitch + 16u * (slot ^ ((n >> 2) & 3));
    }
    // scales: wavefronts 0 .. SW - 1, two 32-channel parts each, 8 outputs per lane; zero
    // points: the wavefronts after them, 4 bits: two parts each, 8 outputs per lane, 8 bits:
    // both parts, 16 outputs per lane and half a wavefront
    const int h = lane >> 5;
    part = wave < SW ? 2 * wave + h : BITS == 4 ? 2 * (wave - SW) + h : (lane >> 4) & 1;
    s_ptr = l.scales + min(n0 + 8 * (lane & 31), N - 8);
    const int zn = BITS == 4 ? min(n0 / 8 + (lane & 31), N / 8 - 1) : min(n0 / 4 + 4 * (lane & 15), N / 4 - 4);
    z_ptr = l.zeros.words + (l.zeros.sym ? 0 : zn);
    z_pitch = l.zeros.sym ? 0 : N / (32 / BITS);
  }

  // Stage t to memory t % COUNT; past the end the last one again.  Channels past K (the last
  // stage of K % 128 = 64) are read from within the buffers and not used.
  __device__ __forceinline__ void load(int t) const {
    const uint32_t stage = ring + (t % L::COUNT) * L::BYTES;
    const int tc = min(t, KT - 1);
    const int g = min(tc * BK + 32 * part, K - 1) >> gshift;
    const uint32_t scales = stage + L::A + L::C, zeros = scales + L::S;
    if (wave < SW)
      direct_load<16>(s_ptr + static_cast<size_t>(g) * s_pitch, scales + wave * 1024);
    else if (wave < 2 * SW)
      direct_load<BITS == 4 ? 4 : 16>(z_ptr + static_cast<size_t>(g) * z_pitch, BITS == 4 ? zeros + (wave - SW) * 256 : zeros);
    direct_loads16<AL, 512 * 16>(xr, stage + wave * 1024, a_off, tc * (BK * 2));
    direct_loads16<2, 512 * 16>(qr, stage + L::A + wave * 1024, b_off, tc * 64);
  }

  // Waits for this wavefront's loads of all but the newest COUNT - 2 stages.
  __device__ __forceinline__ void wait() const {
    if (wave < 2 * SW)
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"((L::COUNT - 2) * (AL + 3)) : "memory");
    else
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"((L::COUNT - 2) * (AL + 2)) : "memory");
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
  constexpr int CPR = L::BK / 8;
  const int lane = tid & 63, lc = lane & 31, lh = lane >> 5;
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc.b[b][r] = 0.f;
  const int col = wave * 32 + lc;
  const int a_swz = lc & (CPR - 1), c_swz = (col >> 2) & 3;
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
    const unsigned char* rows = st + lc * L::ROW;
    const unsigned char* codes = st + L::A + col * 64;
#pragma unroll
    for (int v = 0; v < L::BK / 64; ++v) {   // 64 channels at a time
      if (v > 0 && t * L::BK + 64 * v >= ld.K) break;
      uint4 cw[BITS / 4];   // 4 bits: part 2 v + h; 8 bits: parts 2 h and 2 h + 1
      if constexpr (BITS == 4) {
        cw[0] = *reinterpret_cast<const uint4*>(codes + 16 * ((2 * v + lh) ^ c_swz));
      } else {
        cw[0] = *reinterpret_cast<const uint4*>(codes + 16 * ((2 * lh) ^ c_swz));
        cw[1] = *reinterpret_cast<const uint4*>(codes + 16 * ((2 * lh + 1) ^ c_swz));
      }
      if (((t * L::BK + 64 * v) & gmask) == 0) {
        const int half = 2 * v + lh;
        const uint32_t sc = *reinterpret_cast<const uint16_t*>(st + L::A + L::C + (half * 256 + col) * 2);
        const unsigned char* zs = st + L::A + L::C + L::S;
        uint32_t z;
        if constexpr (BITS == 4)
          z = (zeros.word(*reinterpret_cast<const uint32_t*>(zs + (half * 32 + (col >> 3)) * 4)) >> (4 * (lc & 7))) & 0xFu;
        else
          z = zeros.sym ? 128u : *(zs + half * 256 + col);
        dc = make_consts(z, __builtin_bit_cast(half_t, static_cast<uint16_t>(sc)));
      }
      half8_t af[2][RB];
#pragma unroll
      for (int b = 0; b < RB; ++b)
        af[0][b] = *reinterpret_cast<const half8_t*>(rows + 32 * L::ROW * b + 16 * ((8 * v + 4 * lh) ^ a_swz));
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (s < 3) {
#pragma unroll
          for (int b = 0; b < RB; ++b)
            af[(s + 1) & 1][b] =
                *reinterpret_cast<const half8_t*>(rows + 32 * L::ROW * b + 16 * ((8 * v + 4 * lh + s + 1) ^ a_swz));
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
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");   // the clamped loads past the last stage
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
      const float v[1] = {acc.b[b][r]};
      half_t o[1];
      value(32 * b + row, 32 * wave + lc, 32, v, o);
      turn[row * PITCH + lc] = o[0];
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
      acc, smem, tid, RoundValues(),
      [&](int row, int col, half8_t v) {
        if (row < rows && n0 + col < N) *reinterpret_cast<half8_t*>(y + static_cast<size_t>(slots[row]) * N + n0 + col) = v;
      });
}

// experts_gemm_kernel for plans of 64-row tiles.
template <int BITS>
__global__ __launch_bounds__(512, 4) void experts_low_kernel(const half_t* __restrict__ x, int x_rows, int gathered, int S,
                                                             int T, Layers layers, SlotPlan plan, half_t* __restrict__ y) {
  extern __shared__ __align__(16) unsigned char smem[];
  const int tid = threadIdx.x, N = layers.N;
  each_empty(plan, S, [&](int slot) {
    for (int n = 8 * tid; n < N; n += 8 * 512) *reinterpret_cast<half8_t*>(y + static_cast<size_t>(slot) * N + n) = half8_t{};
  });
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
  const Layers l = layers.at<BITS>(tile.expert);
  if (tile.rows > 32)
    low_tile<2, BITS>(x, x_rows, l, y, smem, source, slots, tile.rows, n0);
  else
    low_tile<1, BITS>(x, x_rows, l, y, smem, source, slots, tile.rows, n0);
}

}  // namespace w4a16
