// What the grouped products share: slots (a row of the batch and one of its experts) grouped
// by expert, the list of row tiles over them, and the experts' packed layers.
//
// The sizes of the groups are known only on the device, so the products run over a list of
// row tiles that plan_slots_kernel makes there: up to 256 slots of one expert, the remainder
// of an expert in the smallest tile of 64, 128 or 256 rows that holds it (a product of 64
// rows costs well below half of the 256-row one).
#pragma once

#include "nibbles.hpp"

namespace w4a16 {

constexpr int kMaxExperts = 512;
constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kPanelTiles = 4;   // row tiles of an expert that take the same weight columns in turn

struct RowTile {
  int32_t expert;        // -1: slots without an expert
  int32_t first;         // place of its first slot in the order
  int32_t rows;          // slots, at most `height`
  int32_t height;        // 64, 128 or 256
  int32_t panel_first;   // its panel: up to kPanelTiles tiles of one expert
  int32_t panel_tiles;
  int32_t pad[2];
};

struct SlotPlan {
  int32_t* counts;   // [0] tiles, [1] slots with an expert
  int32_t* order;    // [S] slots by expert
  RowTile* tiles;
};

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

// Where the sums of a transposed product go: out (binary16, one part and one slot per row):
// rounded once, dx0 added; else partial sums part[split][row][K] in fp32, added to what is
// there where `add` is set.
struct TOut {
  half_t* out;
  const half_t* dx0;
  float* part;
  size_t part_rows;
  int add;
};

}  // namespace w4a16
