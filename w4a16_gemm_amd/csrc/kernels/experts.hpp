// Products grouped by expert: y[slot] = x[slot / T] W^_e^T, a workgroup per row tile of the
// plan and 256 (64 NB) output channels, results to the slots' rows of y.  Tiles of 256 rows
// take the 16x16x32 product, smaller ones the 32x32x16 product (tile.hpp).
#pragma once

#include "tile.hpp"

namespace w4a16 {

// Stores a tile of accumulators as binary16: value(row, column, step, v, o) makes the binary16
// values o of v in the tile's row and columns `column`, `column` + step and so on, put(row,
// column, run of 8 columns) stores them.  An accumulator register
// holds 16 (32) neighbouring columns of a row, 32 (64) bytes; to store whole 128-byte runs a
// wavefront turns 32 rows at a time in LDS memory of its own (rows of 16 NB columns and 16
// bytes of padding, so that the rows that one write meets lie in distinct banks).  The ring's
// memory is used: every wavefront must be done with its loads.
template <int NB>
constexpr int turn_pitch() { return 16 * NB + 8; }

template <int NB, int MB, class Put>
__device__ __forceinline__ void put_turned(const half_t* turn, int tid, int row0, Put put) {
  const int lane = tid & 63, wn = (tid >> 6) & 3;
  constexpr int RUNS = 2 * NB;   // runs of 8 columns per row
#pragma unroll
  for (int i = 0; i < 32 * RUNS / 64; ++i) {
    const int at = i * 64 + lane, row = at / RUNS, run = at % RUNS;
    put(row0 + row, wn * 16 * NB + 8 * run, *reinterpret_cast<const half8_t*>(turn + row * turn_pitch<NB>() + 8 * run));
  }
}

template <int NB, int MB, class Value, class Put>
__device__ __forceinline__ void store_tile(const float4_t (&acc)[MB][NB], unsigned char* smem, int tid, Value value,
                                           Put put) {
  const int lane = tid & 63, wave = tid >> 6, wm = wave >> 2, wn = wave & 3, lr = lane & 15, lq = lane >> 4;
  half_t* turn = reinterpret_cast<half_t*>(smem) + wave * 32 * turn_pitch<NB>();
#pragma unroll
  for (int m2 = 0; m2 < MB / 2; ++m2) {
    const int row0 = wm * 16 * MB + 32 * m2;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float v[NB];
        half_t o[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) v[nb] = acc[2 * m2 + h][nb][r];
        value(row0 + 16 * h + 4 * lq + r, wn * 16 * NB + lr, 16, v, o);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) turn[(16 * h + 4 * lq + r) * turn_pitch<NB>() + 16 * nb + lr] = o[nb];
      }
    put_turned<NB, MB>(turn, tid, row0, put);
  }
}

template <int NB, int MB, class Value, class Put>
__device__ __forceinline__ void store_tile32(const f32x16_t (&acc)[MB / 2][NB / 2], unsigned char* smem, int tid,
                                             Value value, Put put) {
  const int lane = tid & 63, wave = tid >> 6, wm = wave >> 2, wn = wave & 3, lc = lane & 31, lh = lane >> 5;
  half_t* turn = reinterpret_cast<half_t*>(smem) + wave * 32 * turn_pitch<NB>();
#pragma unroll
  for (int rb = 0; rb < MB / 2; ++rb) {
    const int row0 = wm * 16 * MB + 32 * rb;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int row = 8 * (r >> 2) + 4 * lh + (r & 3);
      float v[NB / 2];
      half_t o[NB / 2];
#pragma unroll
      for (int cb = 0; cb < NB / 2; ++cb) v[cb] = acc[rb][cb][r];
      value(row0 + row, wn * 16 * NB + lc, 32, v, o);
#pragma unroll
      for (int cb = 0; cb < NB / 2; ++cb) turn[row * turn_pitch<NB>() + 32 * cb + lc] = o[cb];
    }
    put_turned<NB, MB>(turn, tid, row0, put);
  }
}

struct RoundValues {
  template <int COUNT>
  __device__ __forceinline__ void operator()(int, int, int, const float (&v)[COUNT], half_t (&o)[COUNT]) const {
#pragma unroll
    for (int i = 0; i < COUNT; ++i) o[i] = static_cast<half_t>(v[i]);
  }
};

template <int NB, int MB, int BITS, int BM>
__device__ __forceinline__ void experts_tile(const half_t* x, int x_rows, const Layers& l, half_t* y, unsigned char* smem,
                                             const int32_t* source, const int32_t* slots, int rows, int n0) {
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const TileLoader<NB, MB, BITS, BM> ld(x, x_rows, l, smem, source, rows, n0, tid, wave);
  const int N = l.N;
  const RoundValues value;
  auto put = [&](int row, int col, half8_t v) {
    if (row < rows && n0 + col < N) *reinterpret_cast<half8_t*>(y + static_cast<size_t>(slots[row]) * N + n0 + col) = v;
  };
  if constexpr (MB < 8 && NB % 2 == 0) {
    f32x16_t acc[MB / 2][NB / 2];
    tile_product32(ld, l.zeros, smem, tid, wave, acc);
    __syncthreads();
    store_tile32<NB, MB>(acc, smem, tid, value, put);
  } else {
    float4_t acc[MB][NB];
    tile_product(ld, l.zeros, smem, tid, wave, acc);
    __syncthreads();
    store_tile<NB, MB>(acc, smem, tid, value, put);
  }
}

// gathered: x holds the valid slots' rows in the plan's order (act order), else row m of x
// is that of slots [m T, (m + 1) T).
// BM: of tile.hpp, at least the plan's height.
template <int NB, int BITS, int BM>
__global__ __launch_bounds__(512, BM == 256 ? 2 : 4) void experts_gemm_kernel(const half_t* __restrict__ x, int x_rows, int gathered, int S,
                                                           int T, Layers layers, SlotPlan plan, half_t* __restrict__ y) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int BN = 64 * NB;
  const int tid = threadIdx.x, N = layers.N;
  each_empty(plan, S, [&](int slot) {
    for (int n = 8 * tid; n < N; n += 8 * 512) *reinterpret_cast<half8_t*>(y + static_cast<size_t>(slot) * N + n) = half8_t{};
  });
  RowTile tile;
  int col;
  if (!find_tile(plan, (N + BN - 1) / BN, blockIdx.x, tile, col)) return;
  int32_t* slots = reinterpret_cast<int32_t*>(smem + tile_lds<BITS, BM>() - 16 * BM);
  int32_t* source = slots + BM;
  if (tid < tile.rows) {
    const int s = plan.order[tile.first + tid];
    slots[tid] = s;
    source[tid] = gathered ? tile.first + tid : s / T;
  }
  __syncthreads();
  const int n0 = col * BN;
  const Layers l = layers.at<BITS>(tile.expert);
  if (BM == 256 && tile.height == 256)
    experts_tile<NB, BM == 256 ? 8 : 4, BITS, BM>(x, x_rows, l, y, smem, source, slots, tile.rows, n0);
  else if (tile.height == 128)
    experts_tile<NB, 4, BITS, BM>(x, x_rows, l, y, smem, source, slots, tile.rows, n0);
  else
    experts_tile<NB, 2, BITS, BM>(x, x_rows, l, y, smem, source, slots, tile.rows, n0);
}

}  // namespace w4a16
