// What the grouped products share: slots (a row of the batch and one of its experts) grouped
// by expert, the list of row tiles over them, and the experts' packed layers.
//
// The sizes of the groups are known only on the device, so the products run over a list of
// row tiles that is made there (slots.hpp): up to `height` slots of one expert, 64, 128 or 256
// by the call's sizes, the remainder of an expert in the smallest tile up to that height that
// holds it (a product of 64 rows costs well below half of the 256-row one).
#pragma once

#include "nibbles.hpp"
#include "parts.hpp"

namespace w4a16 {

constexpr int kMaxExperts = 512;
constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kPanelTiles = 4;   // row tiles of an expert that take the same weight columns in turn

struct RowTile {
  int32_t expert;
  int32_t first;         // place of its first slot in the order
  int32_t rows;          // slots, at most `height`
  int32_t height;        // 64, 128 or 256, at most the plan's
  int32_t panel_first;   // its panel: up to kPanelTiles tiles of one expert
  int32_t panel_tiles;
  int32_t pad[2];
};

struct SlotPlan {
  int32_t* counts;   // [0] tiles, [1] slots with an expert
  int32_t* order;    // [S] slots by expert, those without one last
  RowTile* tiles;
  int32_t* tile_of;  // [S] tile of every slot with an expert, or NULL: not needed
  int32_t* sums;     // while it is made, see plan_blocks
};

// Workgroups that make a plan: one for up to kPlanSlots slots, else one for every 2048 slots, at
// most 256.
constexpr int kPlanSlots = 16384;
inline int plan_blocks(int64_t S) {
  const int64_t blocks = (S + 2047) / 2048;
  return S <= kPlanSlots ? 1 : blocks < 256 ? static_cast<int>(blocks) : 256;
}

__host__ __device__ inline int rest_height(int rows, int height) {
  return rows <= 64 ? 64 : rows <= 128 && height > 128 ? 128 : height;
}

// The packed layers of E experts (or one layer), the weights of one after the other.
struct Layers {
  const uint32_t* qw;
  const half_t* scales;
  Zeros zeros;
  size_t words;   // per expert, the act-order tail included
  int N, K, gshift, G;

  template <int BITS>
  __device__ __forceinline__ Layers at(int e) const {
    Layers l = *this;
    l.qw += static_cast<size_t>(e) * words;
    l.scales += static_cast<size_t>(e) * G * N;
    if (!zeros.sym) l.zeros.words += static_cast<size_t>(e) * G * (N / (32 / BITS));
    return l;
  }
  // stored position -> input channel of an expert (act order)
  __device__ __forceinline__ const int32_t* order(int e) const {
    return reinterpret_cast<const int32_t*>(qw + static_cast<size_t>(e + 1) * words - K);
  }
};

// The row tile and column tile of this workgroup, of counts[0] x tiles_n.  Workgroups go
// round-robin to the 8 XCDs; each XCD takes a contiguous run of the tiles, panel by panel,
// the row tiles of a panel before the next columns, so that the rows of a panel and the
// weight columns in use stay in its L2.  False: no tile is left for this workgroup.
__device__ __forceinline__ bool find_tile(const SlotPlan& plan, int tiles_n, int bid, RowTile& tile, int& col) {
  const int total = plan.counts[0] * tiles_n;
  const int chunk = (total + 7) >> 3;
  const int id = (bid & 7) * chunk + (bid >> 3);
  if ((bid >> 3) >= chunk || id >= total) return false;
  const RowTile any = plan.tiles[id / tiles_n];
  const int local = id - any.panel_first * tiles_n;
  tile = plan.tiles[any.panel_first + local % any.panel_tiles];
  col = local / any.panel_tiles;
  return true;
}

// The slots without an expert, shared out over all workgroups: what is written there takes
// none of the tiles' turns (as tiles in the list they filled some XCDs' runs and left others
// with more than their share of products: 820 of 1641 slots on three experts, K 7808, N 10112
// 642 us, so 379 us).
template <class F>
__device__ __forceinline__ void each_empty(const SlotPlan& plan, int S, F f) {
  for (int64_t p = static_cast<int64_t>(plan.counts[1]) + blockIdx.x; p < S; p += gridDim.x) f(plan.order[p]);
}

// Workgroups of an XCD (32 compute units) that run at once, by the rows that a tile's memory has
// room for.
__host__ __device__ constexpr int tile_slots(int bm) { return bm == 256 ? 32 : 64; }

// Products of too few tiles for whole rounds over the compute units: each XCD (`side` workgroups
// at once) takes `chunk` tiles, whole rounds of them as they are, the rest each in `pieces` parts
// of the contraction, as many as make the rest's rounds shortest (parts.hpp).
// Measured, whole calls: a training batch of 8192 slots over eight 8-bit experts (K 4096, N
// 14336; about 36 row tiles of 16 columns, 2.25 rounds) 1683 -> 1348 us; 777 rows of two of
// eight act-order experts of group 32 405 -> 361 us.
struct Pieces {
  int chunk, whole, pieces;

  __device__ __forceinline__ Pieces(int total, int most, int side, int outputs) {
    chunk = (total + 7) >> 3;
    const int rest = chunk % side;
    whole = chunk - rest;
    pieces = parts_of(rest, most, side, outputs);
  }
  // parts of tile id
  __device__ __forceinline__ int of(int id) const { return id % chunk < whole ? 1 : pieces; }
  // parts of a row tile's column
  __device__ __forceinline__ int of(const RowTile& t, int tile, int col, int cols) const {
    return of(t.panel_first * cols + col * t.panel_tiles + tile - t.panel_first);
  }
};

// Workgroups that cover every part: 8 ((most chunk rounded down to `side`) + 2 side).
__host__ __device__ inline int64_t piece_blocks(int64_t tiles, int side) { return 8 * ((tiles + 7) / 8 / side * side + 2 * side); }

// The row tile, column and part of this workgroup; see find_tile.
__device__ __forceinline__ bool find_piece(const SlotPlan& plan, int cols, int most, int side, int outputs, int bid, RowTile& tile, int& col,
                                           int& piece, int& pieces) {
  const int total = plan.counts[0] * cols;
  if (total == 0) return false;
  const Pieces rule(total, most, side, outputs);
  const int j = bid >> 3;
  int local = j;
  piece = 0, pieces = 1;
  if (j >= rule.whole) {
    pieces = rule.pieces;
    local = rule.whole + (j - rule.whole) / pieces;
    piece = (j - rule.whole) % pieces;
  }
  const int id = (bid & 7) * rule.chunk + local;
  if (local >= rule.chunk || id >= total) return false;
  const RowTile any = plan.tiles[id / cols];
  const int at = id - any.panel_first * cols;
  tile = plan.tiles[any.panel_first + at % any.panel_tiles];
  col = at / any.panel_tiles;
  return true;
}

// Where the sums of a transposed product go: a tile that is not in parts to out (binary16,
// one slot per row), rounded once, dx0 added; else (out NULL, or a tile in parts) to the
// partial sums part[piece][row][K] in fp32, added to what is there where `add` is set.
struct TOut {
  half_t* out;
  const half_t* dx0;
  float* part;
  size_t part_rows;
  int add;
};

}  // namespace w4a16
