// Products through the frozen weights the other way: dx[row] = sum_n dy[row][n] W^[n][k],
// straight from the packed codes, which lie along k while the contraction runs along n.
//
// A workgroup of 8 wavefronts (2 along the rows x 4 along k) takes a tile of BM = 32 MB
// rows by 256 channels k, the contraction in tiles of 64 outputs n through an LDS
// ring filled by direct-to-LDS loads ahead of its use, as in the forward tile:
//  * dy: BM rows of 8 chunks of 8 outputs, chunk j of row r at slot j ^ (r / 2 % 8);
//  * codes: 64 rows n of 256 channels, as they lie in memory, in 8 chunks of 8 rows; a
//    chunk is followed by 32 bytes (64 at 8 bits) of padding, so that the four chunks that
//    one MFMA operand reads lie in distinct banks;
//  * scales and zero points of the groups of the tile's eight 32-channel columns.
// The transposition costs one v_perm per two words.  Lane (r, q) of a wavefront reads, for
// the 8 outputs n of chunk j = 4 s + q of MFMA step s, the word of its channels: 4 bits: the
// channels [8 (r % 8), +8) of the wavefront's 64, of which lanes r < 8 take the even ones and
// the others the odd ones.  Even channels sit in the low half of a word and odd ones in the
// high half (nibbles.hpp), so one v_perm of the words of outputs n and n + 1 gives a register
// whose nibble i holds the codes of channel 2 i (+ 1) for both outputs, and the same masks as
// in the forward product turn it into pairs along n.  Block i = 0..3 of the wavefront then has
// the channels 8 (r % 8) + 2 i + r / 8.  8 bits: lane r takes the word of channels
// [4 r, +4), one v_perm per pair and channel; block i has the channels 4 r + i.
// The weights are binary16((q - Z) S), the values of the forward product.
// VALU work per MFMA is that of the forward product plus the v_perm and the zero points'
// constants, which here change with every output n instead of staying with the lane.
#pragma once

#include "tile.hpp"

namespace w4a16 {

template <int BITS, int BM>
struct TStage {
  static constexpr uint32_t ROW = 256 * BITS / 8;                 // code bytes of a row
  static constexpr uint32_t CHUNK = 8 * ROW + (BITS == 4 ? 32 : 64);
  static constexpr uint32_t A = BM * 64 * 2;
  static constexpr uint32_t C = 8 * CHUNK;
  static constexpr uint32_t S = 8 * 64 * 2;                       // [column / 32][output]
  static constexpr uint32_t Z = BITS == 4 ? 256 : 1024;           // [column / 32][output], 64 lanes' loads
  static constexpr uint32_t BYTES = A + C + S + Z;
  static constexpr int COUNT = BITS == 8 && BM == 128 ? 2 : 3;    // as in TileStage
  static_assert(BYTES % 16 == 0, "stage alignment");
};

// Behind the ring: a word per row of the tile.
template <int BITS, int BM>
constexpr size_t transposed_lds() { return TStage<BITS, BM>::COUNT * static_cast<size_t>(TStage<BITS, BM>::BYTES) + 4 * BM; }
static_assert(transposed_lds<4, 256>() <= 160 * 1024 && transposed_lds<8, 256>() <= 160 * 1024, "fits a compute unit");
static_assert(transposed_lds<4, 128>() <= 80 * 1024 && transposed_lds<8, 128>() <= 80 * 1024, "two workgroups per compute unit");

// Loads of one tile: rows source[0 .. rows) of a [a_rows][a_pitch] from column a0 on against
// the outputs [n_begin, n_end) and the channels from k0 on.
template <int MB, int BITS, int BM>
struct TLoader {
  using L = TStage<BITS, BM>;
  static constexpr int APT = 32 * MB / 64;   // activation chunks (16 B) per thread and stage
  static constexpr int CL = BITS / 4;        // code loads per thread and stage

  u32x4_t ar, qr;
  const half_t* s_ptr;      // this lane's scales of tile 0 (wavefront 0)
  const uint32_t* z_ptr;    // this lane's zero points of tile 0 (wavefront 1)
  uint32_t ring;            // LDS offset
  int KT, wave, s_step, z_step, s_tail, z_tail;
  uint32_t a_off[APT], b_off[CL], b_tail[CL], b_step;

  __device__ __forceinline__ TLoader(const half_t* a, int a_rows, int a_pitch, int a0, const Layers& l, int n_begin,
                                     int n_end, int k0, const int32_t* source, int rows, unsigned char* smem_, int tid,
                                     int wave_)
      : ring(lds_offset(smem_)), KT((n_end - n_begin + 63) / 64), wave(wave_) {
    const int lane = tid & 63;
    const uint32_t pitch = static_cast<uint32_t>(l.K) * BITS / 8;   // code bytes of a row
    ar = direct_rsrc(a + a0, (static_cast<uint32_t>(a_rows) * a_pitch - a0) * 2u);
    qr = direct_rsrc(reinterpret_cast<const unsigned char*>(l.qw) + static_cast<size_t>(n_begin) * pitch,
                     static_cast<uint32_t>(n_end - n_begin) * pitch);
#pragma unroll
    for (int i = 0; i < APT; ++i) {
      const int c = (wave * APT + i) * 64 + lane;
      const int row = c >> 3, slot = c & 7;
      a_off[i] = (static_cast<uint32_t>(source[min(row, rows - 1)]) * a_pitch + 8 * (slot ^ ((row >> 1) & 7))) * 2u;
    }
    // Codes: load i of wavefront w fills rows 8 w .. (4 bits: 8 rows, 8 bits: 4 rows each),
    // 16 bytes per lane; channels past K re-read the row's last ones, outputs past the end
    // the last one (their dy is masked).
    constexpr int PIECES = L::ROW / 16;
    const int last = static_cast<int>((n_end - n_begin - 1) % 64);   // last output of the last tile
#pragma unroll
    for (int i = 0; i < CL; ++i) {
      const int row = 8 * wave + (i * 64 + lane) / PIECES, piece = lane % PIECES;
      const uint32_t col = min(static_cast<uint32_t>(k0) * BITS / 8 + 16 * piece, pitch - 16);
      b_off[i] = static_cast<uint32_t>(row) * pitch + col;
      b_tail[i] = static_cast<uint32_t>(min(row, last)) * pitch + col;
    }
    b_step = 64 * pitch;
    // Scales: lane = 8 (column / 32) + piece of 8 outputs.  Zero points: 4 bits, lane = 8
    // (column / 32) + word of 8 outputs; 8 bits, lane = 4 (column / 32) + piece of 16 outputs
    // (the upper lanes fill 512 bytes behind them again).
    auto group = [&](int c32) { return min(k0 + 32 * c32, l.K - 1) >> l.gshift; };
    const int sp = 8 * (lane & 7);
    s_ptr = l.scales + static_cast<size_t>(group(lane >> 3)) * l.N + n_begin + sp;
    s_step = 64;
    s_tail = min(sp, last / 8 * 8) - sp;
    constexpr int ZP = BITS == 4 ? 8 : 16;   // outputs per zero-point load of a lane
    const int zl = BITS == 4 ? lane : lane & 31;
    const int zp = ZP * (zl % (64 / ZP));
    const size_t z_at = (static_cast<size_t>(group(zl / (64 / ZP))) * l.N + n_begin + zp) / (32 / BITS);
    z_ptr = l.zeros.words + (l.zeros.sym ? 0 : z_at);
    z_step = l.zeros.sym ? 0 : 64 / (32 / BITS);
    z_tail = l.zeros.sym ? 0 : (min(zp, last / ZP * ZP) - zp) / (32 / BITS);
  }

  // Tile t to stage t % COUNT; tiles past the end re-load the last one.  The scale and zero-point
  // loads come first: waiting for tile t never waits for more than those of tile t + 1.
  __device__ __forceinline__ void load(int t) const {
    const uint32_t stage = ring + (t % L::COUNT) * L::BYTES;
    const int tc = min(t, KT - 1);
    const bool tail = tc == KT - 1;
    const uint32_t scales = stage + L::A + L::C;
    if (wave == 0)
      direct_load<16>(s_ptr + static_cast<ptrdiff_t>(tc) * s_step + (tail ? s_tail : 0), scales);
    else if (wave == 1)
      direct_load<BITS == 4 ? 4 : 16>(z_ptr + static_cast<ptrdiff_t>(tc) * z_step + (tail ? z_tail : 0), scales + L::S);
    direct_loads16<APT, 1024>(ar, stage + wave * APT * 1024, a_off, tc * 128);
    uint32_t codes[CL];
#pragma unroll
    for (int i = 0; i < CL; ++i) codes[i] = tail ? b_tail[i] : b_off[i];
    direct_loads16<CL, 1024>(qr, stage + L::A + wave * L::CHUNK, codes, static_cast<uint32_t>(tc) * b_step);
  }
};

// (zero point of output 2 p, of output 2 p + 1) as 16-bit halves, p = 0..3.
__device__ __forceinline__ void zero_pairs4(uint32_t word, uint32_t (&z)[4]) {
  const uint32_t even = word & 0x0F0F0F0Fu, odd = (word >> 4) & 0x0F0F0F0Fu;
#pragma unroll
  for (int p = 0; p < 4; ++p) z[p] = __builtin_amdgcn_perm(odd, even, 0x0c000c00u | p | ((4u + p) << 16));
}

__device__ __forceinline__ uint32_t perm_bytes(uint32_t hi, uint32_t lo, uint32_t sel) {
  return __builtin_amdgcn_perm(hi, lo, sel);
}

// acc[mb][i]: rows 16 mb + 4 q + reg of the wavefront's 16 MB, block i of its channels.
// HALVED (up to 16 MB rows): the two wavefronts of a channel block take the same rows and half of
// every step's outputs each, so that every weight is expanded once; their sums meet in the
// first of them (wave < 4), the other's are void.  (Two rows on 8 of 27 experts, 7488 outputs
// of 1472 channels, 69 -> 52 us; 68 on 2 of 23 8-bit ones, 10224 of 896, 87 -> 65 us.)
template <bool HALVED, int MB, int BITS, int BM>
__device__ __forceinline__ void transposed_product(const TLoader<MB, BITS, BM>& ld, Zeros zeros, unsigned char* smem,
                                                   int outputs, int tid, int wave, float4_t (&acc)[MB][4]) {
  using L = TStage<BITS, BM>;
  using Loader = TLoader<MB, BITS, BM>;
  constexpr int INFLIGHT = (L::COUNT - 2) * (Loader::APT + Loader::CL);
  const int lane = tid & 63;
  const int wm = wave >> 2, wn = wave & 3;
  const int lr = lane & 15, lq = lane >> 4;
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[mb][i] = float4_t{0.f, 0.f, 0.f, 0.f};

  const uint32_t a_lane = ((HALVED ? 0 : wm * 16 * MB) + lr) * 128;
  const uint32_t c_lane = L::A + lq * L::CHUNK + (BITS == 4 ? wn * 8 + (lr & 7) : wn * 16 + lr) * 4;
  const int c32 = 2 * wn + (BITS == 4 ? (lr & 7) >> 2 : lr >> 3);   // column / 32 of this lane's channels
  const uint32_t s_lane = L::A + L::C + c32 * 128 + lq * 16;
  const uint32_t z_lane = L::A + L::C + L::S + c32 * (8 * BITS) + lq * BITS;
  const uint32_t half_sel = lr & 8 ? 0x07060302u : 0x05040100u;   // high or low halves of two words
  const int last = outputs - (ld.KT - 1) * 64;                    // outputs of the last tile

#pragma unroll
  for (int t = 0; t < L::COUNT - 1; ++t) ld.load(t);
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(INFLIGHT) : "memory");
  block_barrier();

  for (int t = 0; t < ld.KT; ++t) {
    ld.load(t + L::COUNT - 1);
    const unsigned char* st = smem + (t % L::COUNT) * L::BYTES;
#pragma unroll
    for (int turn = 0; turn < (HALVED ? 1 : 2); ++turn) {
      const int s = HALVED ? wm : turn;
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w[i] = *reinterpret_cast<const uint32_t*>(st + c_lane + s * 4 * L::CHUNK + i * L::ROW);
      const uint4 sv = *reinterpret_cast<const uint4*>(st + s_lane + 64 * s);
      uint32_t sc[4] = {sv.x, sv.y, sv.z, sv.w};
      uint32_t z[4];
      if constexpr (BITS == 4) {
        zero_pairs4(zeros.word(*reinterpret_cast<const uint32_t*>(st + z_lane + 16 * s)), z);
      } else {
        const uint2 zw = *reinterpret_cast<const uint2*>(st + z_lane + 32 * s);
        const uint32_t z0 = zeros.word8(zw.x), z1 = zeros.word8(zw.y);
        z[0] = perm_bytes(0, z0, 0x0c010c00u), z[1] = perm_bytes(0, z0, 0x0c030c02u);
        z[2] = perm_bytes(0, z1, 0x0c010c00u), z[3] = perm_bytes(0, z1, 0x0c030c02u);
      }
      half8_t af[MB];
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
        af[mb] = *reinterpret_cast<const half8_t*>(st + a_lane + 16 * ((4 * s + lq) ^ (lr >> 1)) + 2048 * mb);
      if (t == ld.KT - 1) {   // outputs past the end: nothing of dy there, weights of 0
        const int left = last - 8 * (4 * s + lq);
#pragma unroll
        for (int p = 0; p < 4; ++p) sc[p] = 2 * p + 1 < left ? sc[p] : 2 * p < left ? sc[p] & 0xFFFFu : 0u;
        if (left <= 0) {
#pragma unroll
          for (int mb = 0; mb < MB; ++mb) af[mb] = half8_t{};
        }
      }
      uint32_t b[4][4];   // [block][pair of outputs]
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const half2_t n1024 = as_h2(z[p] | 0xE400E400u), scale = as_h2(sc[p]);
        if constexpr (BITS == 4) {
          const half2_t n64 = as_h2((z[p] << 4) | 0xD400D400u);
          const half2_t sixteenth = half2_t{static_cast<half_t>(0.0625f), static_cast<half_t>(0.0625f)};
          const uint32_t v = perm_bytes(w[2 * p + 1], w[2 * p], half_sel);
          const uint32_t u = v >> 8;
          b[0][p] = __builtin_bit_cast(uint32_t, (as_h2(and_or(v, 0x000F000Fu, kMagic)) + n1024) * scale);
          b[1][p] = __builtin_bit_cast(
              uint32_t, __builtin_elementwise_fma(as_h2(and_or(v, 0x00F000F0u, kMagic)), sixteenth, n64) * scale);
          b[2][p] = __builtin_bit_cast(uint32_t, (as_h2(and_or(u, 0x000F000Fu, kMagic)) + n1024) * scale);
          b[3][p] = __builtin_bit_cast(
              uint32_t, __builtin_elementwise_fma(as_h2(and_or(u, 0x00F000F0u, kMagic)), sixteenth, n64) * scale);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {   // element i of a word is its byte 0, 2, 1, 3
            const uint32_t byte = i == 1 ? 2 : i == 2 ? 1 : i;
            const uint32_t v = perm_bytes(w[2 * p + 1], w[2 * p], 0x0c000c00u | byte | ((4 + byte) << 16));
            b[i][p] = __builtin_bit_cast(uint32_t, (as_h2(v | kMagic) + n1024) * scale);
          }
        }
      }
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc[mb][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
              af[mb], __builtin_bit_cast(half8_t, uint4{b[i][0], b[i][1], b[i][2], b[i][3]}), acc[mb][i], 0, 0, 0);
      __builtin_amdgcn_s_setprio(0);
    }
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(INFLIGHT) : "memory");
    block_barrier();
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  if constexpr (HALVED) {
    block_barrier();   // every wavefront's clamped loads have landed
    float4_t* other = reinterpret_cast<float4_t*>(smem) + wn * (MB * 4 * 64) + lane;
    if (wm == 1) {
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int i = 0; i < 4; ++i) other[(4 * mb + i) * 64] = acc[mb][i];
    }
    __syncthreads();
    if (wm == 0) {
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[mb][i] += other[(4 * mb + i) * 64];
    }
  }
}

// Calls store(row, channel, v0..v7 or v0..v3) with consecutive channels: row inside the
// tile, channel from the tile's first.  4 bits: lanes r and r + 8 hold the even and the odd
// channels of the same eight; each gives the other two of its four rows.
template <int MB, int BITS, class Store>
__device__ __forceinline__ void each_run(const float4_t (&acc)[MB][4], int tid, Store store) {
  const int lane = tid & 63, wave = tid >> 6, wm = wave >> 2, wn = wave & 3, lr = lane & 15, lq = lane >> 4;
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) {
    const int row0 = wm * 16 * MB + 16 * mb + 4 * lq;
    if constexpr (BITS == 4) {
      const bool odd = (lr & 8) != 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float keep = odd ? acc[mb][i][2 + h] : acc[mb][i][h];
          const float give = odd ? acc[mb][i][h] : acc[mb][i][2 + h];
          const float got = __builtin_bit_cast(
              float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, give), 0x128, 0xF, 0xF, true));   // lane r ^ 8
          v[2 * i] = odd ? got : keep;
          v[2 * i + 1] = odd ? keep : got;
        }
        store(row0 + (odd ? 2 : 0) + h, wn * 64 + 8 * (lr & 7), v);
      }
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float v[4] = {acc[mb][0][r], acc[mb][1][r], acc[mb][2][r], acc[mb][3][r]};
        store(row0 + r, wn * 64 + 4 * lr, v);
      }
    }
  }
}

template <bool HALVED, int MB, int BITS, int BM>
__device__ __forceinline__ void transposed_tile(const half_t* a, int a_rows, int a_pitch, int a0, const Layers& l,
                                                int n_begin, int n_end, int n_valid, int k0, const int32_t* source,
                                                const RowTile& tile, const TOut& to, int piece, int pieces,
                                                unsigned char* smem) {
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rows = tile.rows;
  float4_t acc[MB][4];
  if (n_begin < n_end) {
    const TLoader<MB, BITS, BM> ld(a, a_rows, a_pitch, a0, l, n_begin, n_end, k0, source, rows, smem, tid, wave);
    transposed_product<HALVED>(ld, l.zeros, smem, min(n_end, n_valid) - n_begin, tid, wave, acc);
  } else {   // a part without outputs: nothing to add
    if (to.add) return;
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[mb][i] = float4_t{0.f, 0.f, 0.f, 0.f};
  }
  if (HALVED && wave >= 4) return;
  const int K = l.K;
  constexpr int RUN = BITS == 4 ? 8 : 4;
  each_run<MB, BITS>(acc, tid, [&](int row, int col, const float* v) {
    if (row >= rows || k0 + col >= K) return;
    if (to.out && pieces == 1) {
      typedef _Float16 run_t __attribute__((ext_vector_type(RUN)));
      const size_t at = static_cast<size_t>(source[row]) * K + k0 + col;
      run_t d{}, o;
      if (to.dx0) d = *reinterpret_cast<const run_t*>(to.dx0 + at);
#pragma unroll
      for (int i = 0; i < RUN; ++i) o[i] = static_cast<half_t>(v[i] + static_cast<float>(d[i]));
      *reinterpret_cast<run_t*>(to.out + at) = o;
    } else {
      float4_t* p = reinterpret_cast<float4_t*>(to.part + (piece * to.part_rows + source[row]) * K + k0 + col);
#pragma unroll
      for (int i = 0; i < RUN / 4; ++i) {
        float4_t s = {v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
        if (to.add) s += p[i];
        p[i] = s;
      }
    }
  });
}

// slots: of the plan.  a [a_rows][a_pitch]: by_place: row p belongs to place p of the plan's order, else row s to
// slot s.  The outputs [n_begin, n_end) against columns [0, n_end - n_begin) of a; those from
// n_valid > n_end - 16 on, whose columns of a are 0, count as 0 whatever their scales.  A tile
// in parts takes ceil(n_most / parts) outputs each, n_most >= n_end - n_begin (the same for
// every launch that adds to the same sums).  Sums go to the places or slots alike.
template <int BITS, int BM>
__global__ __launch_bounds__(512, BM == 256 ? 2 : 4) void transposed_kernel(const half_t* __restrict__ a, int a_rows, int a_pitch,
                                                         int by_place, Layers layers, SlotPlan plan, int slots, int n_begin,
                                                         int n_end, int n_valid, int n_most, int most, TOut to) {
  extern __shared__ __align__(16) unsigned char smem[];
  const int tid = threadIdx.x, K = layers.K;
  if (to.out)   // slots without an expert: dx0 alone
    each_empty(plan, slots, [&](int slot) {
      for (int k = 8 * tid; k < K; k += 8 * 512) {
        const size_t at = static_cast<size_t>(slot) * K + k;
        *reinterpret_cast<half8_t*>(to.out + at) = to.dx0 ? *reinterpret_cast<const half8_t*>(to.dx0 + at) : half8_t{};
      }
    });
  RowTile tile;
  int col, piece, pieces;
  if (!find_piece(plan, (K + 255) / 256, most, tile_slots(BM), n_most, blockIdx.x, tile, col, piece, pieces)) return;
  const int k0 = col * 256;
  int32_t* rows = reinterpret_cast<int32_t*>(smem + transposed_lds<BITS, BM>() - 4 * BM);
  if (tid < tile.rows) rows[tid] = by_place ? tile.first + tid : plan.order[tile.first + tid];
  __syncthreads();
  const Layers l = layers.at<BITS>(tile.expert);
  const int len = (n_most + 64 * pieces - 1) / (64 * pieces) * 64;
  const int a0 = piece * len, n0 = n_begin + a0, n1 = min(n_end, n0 + len);
  if (BM == 256 && tile.height == 256)
    transposed_tile<false, BM == 256 ? 8 : 4, BITS, BM>(a, a_rows, a_pitch, a0, l, n0, n1, n_valid, k0, rows, tile, to, piece, pieces, smem);
  else if (tile.height == 128)
    transposed_tile<false, 4, BITS, BM>(a, a_rows, a_pitch, a0, l, n0, n1, n_valid, k0, rows, tile, to, piece, pieces, smem);
  else if (tile.rows <= 32)
    transposed_tile<true, 2, BITS, BM>(a, a_rows, a_pitch, a0, l, n0, n1, n_valid, k0, rows, tile, to, piece, pieces, smem);
  else
    transposed_tile<false, 2, BITS, BM>(a, a_rows, a_pitch, a0, l, n0, n1, n_valid, k0, rows, tile, to, piece, pieces, smem);
}

// Partial sums part[piece][slot][K] of the slots [m T, (m + 1) T) -> dx[m], in a fixed
// order, plus dx0, rounded once.  Slots without an expert have no sums.
struct SlotSums {
  const float* part;
  size_t slots;
  const SlotPlan& plan;
  Pieces rule;
  int K, cols, E;

  // adds the parts of one slot at channels [k, k + 8); false: its tile was not in parts
  __device__ __forceinline__ bool add(size_t slot, int tile, const RowTile& row, int k, bool direct, float (&s)[8]) const {
    const int pieces = rule.of(row, tile, k / 256, cols);
    if (direct && pieces == 1) return false;
#pragma unroll 4
    for (int p = 0; p < pieces; ++p) {
      const float* at = part + (p * slots + slot) * K + k;
      const float4_t lo = *reinterpret_cast<const float4_t*>(at), hi = *reinterpret_cast<const float4_t*>(at + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] += lo[i], s[4 + i] += hi[i];
    }
    return true;
  }
};

__device__ __forceinline__ void start_sums(const half_t* dx0, float (&s)[8]) {
  half8_t d = {};
  if (dx0) d = *reinterpret_cast<const half8_t*>(dx0);
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = static_cast<float>(d[i]);
}
__device__ __forceinline__ void store_sums(const float (&s)[8], half_t* out) {
  half8_t o;
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = static_cast<half_t>(s[i]);
  *reinterpret_cast<half8_t*>(out) = o;
}

// direct: tiles that are not in parts have been written already.
__global__ __launch_bounds__(256) void sum_slots_kernel(const float* __restrict__ part, size_t slots, int most, int side, int outputs, int T,
                                                        const int32_t* __restrict__ index, int E, SlotPlan plan, int K,
                                                        int direct, const half_t* __restrict__ dx0, half_t* __restrict__ out) {
  const size_t m = blockIdx.x;
  const int cols = (K + 255) / 256;
  const SlotSums sums{part, slots, plan, Pieces(plan.counts[0] * cols, most, side, outputs), K, cols, E};
  for (int k = 8 * threadIdx.x; k < K; k += 8 * 256) {
    float s[8];
    start_sums(dx0 ? dx0 + m * K + k : nullptr, s);
    bool any = !direct;
    for (int t = 0; t < T; ++t) {
      const size_t slot = m * T + t;
      const int e = index ? index[slot] : 0;
      if (e < 0 || e >= E) continue;
      const int tile = plan.tile_of[slot];
      any |= sums.add(slot, tile, plan.tiles[tile], k, direct != 0, s);
    }
    if (any) store_sums(s, out + m * K + k);
  }
}

// The same with the sums in the stored channel order of each slot's expert (act order):
// inverse [E][K] has the stored position of every channel.  kSumChannels positions at a time
// pass through LDS and are picked up there for kSumChannels channels, so up to that K every
// sum is read once, in order (1554 slots of 4096 channels in two parts: picked up from memory
// 74 us, 20 us).
constexpr int kSumChannels = 8192;

__global__ __launch_bounds__(512) void sum_ordered_kernel(const float* __restrict__ part, size_t slots, int most, int side, int outputs, int T,
                                                          const int32_t* __restrict__ index, int E, SlotPlan plan,
                                                          const int32_t* __restrict__ inverse, int K,
                                                          const half_t* __restrict__ dx0, half_t* __restrict__ out) {
  constexpr int PASS = 8 * 512, RUNS = kSumChannels / PASS;
  __shared__ __align__(16) float turn[kSumChannels];
  const size_t m = blockIdx.x;
  const int cols = (K + 255) / 256, k0 = 8 * threadIdx.x;
  const SlotSums sums{part, slots, plan, Pieces(plan.counts[0] * cols, most, side, outputs), K, cols, E};
  for (int base = 0; base < K; base += kSumChannels) {
    float s[RUNS][8];
#pragma unroll
    for (int r = 0; r < RUNS; ++r) {
      const int k = base + PASS * r + k0;
      start_sums(dx0 && k < K ? dx0 + m * K + k : nullptr, s[r]);
    }
    for (int t = 0; t < T; ++t) {
      const size_t slot = m * T + t;
      const int e = index ? index[slot] : 0;
      if (e < 0 || e >= E) continue;
      const int tile = plan.tile_of[slot];
      const RowTile row = plan.tiles[tile];
      uint4 at[RUNS][2];   // stored positions of the thread's channels
#pragma unroll
      for (int r = 0; r < RUNS; ++r) {
        const int k = min(base + PASS * r + k0, K - 8);
        const uint4* from = reinterpret_cast<const uint4*>(inverse + static_cast<size_t>(e) * K + k);
        at[r][0] = from[0], at[r][1] = from[1];
      }
      for (int c = 0; c < K; c += kSumChannels) {
        const int end = min(K - c, kSumChannels);
        float v[RUNS][8] = {};
#pragma unroll
        for (int r = 0; r < RUNS; ++r)
          if (PASS * r + k0 < end) sums.add(slot, tile, row, c + PASS * r + k0, false, v[r]);
        __syncthreads();   // the last positions are picked up
#pragma unroll
        for (int r = 0; r < RUNS; ++r)
          if (PASS * r + k0 < end) {
            float4_t* to = reinterpret_cast<float4_t*>(turn + PASS * r + k0);
            to[0] = float4_t{v[r][0], v[r][1], v[r][2], v[r][3]};
            to[1] = float4_t{v[r][4], v[r][5], v[r][6], v[r][7]};
          }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < RUNS; ++r) {
          const uint32_t a[8] = {at[r][0].x, at[r][0].y, at[r][0].z, at[r][0].w, at[r][1].x, at[r][1].y, at[r][1].z, at[r][1].w};
          if (base + PASS * r + k0 < K) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (a[i] - c < static_cast<uint32_t>(end)) s[r][i] += turn[a[i] - c];   // not a permutation: left out
          }
        }
      }
    }
#pragma unroll
    for (int r = 0; r < RUNS; ++r) {
      const int k = base + PASS * r + k0;
      if (k < K) store_sums(s[r], out + m * K + k);
    }
  }
}

}  // namespace w4a16
