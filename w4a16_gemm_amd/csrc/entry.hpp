// Host-side helpers of the entry points of the mixtures of experts and of the vocabulary
// head: argument checks, workspace and launches.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "internal.hpp"
#include "kernels/plan.hpp"

namespace w4a16 {
namespace {

int check_launch(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e == hipSuccess) return W4A16_OK;
  return fail(W4A16_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

// The library's error cleared, and the runtime's last-error state, which may hold a
// failure of someone else's call.
void begin_call() {
  clear_error();
  (void)hipGetLastError();
}

struct Buffer {
  const void* ptr;
  uintptr_t align;
  bool required;
  const char* name;
};

template <int COUNT>
int check_buffers(const Buffer (&bufs)[COUNT]) {
  for (const Buffer& b : bufs)
    if (b.required && !b.ptr) return fail(W4A16_ERR_INVALID_ARG, "NULL buffer %s", b.name);
  for (const Buffer& b : bufs)
    if (b.ptr && (reinterpret_cast<uintptr_t>(b.ptr) & (b.align - 1)) != 0)
      return fail(W4A16_ERR_MISALIGNED, "buffer %s is not %d-byte aligned", b.name, static_cast<int>(b.align));
  return W4A16_OK;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Hands out 256-byte aligned pieces of the workspace; with base NULL it only adds them up,
// which is how the _workspace functions know the size.
struct Carver {
  unsigned char* base;
  size_t used = 0;
  template <typename T>
  T* take(size_t count) {
    T* p = base ? reinterpret_cast<T*>(base + used) : nullptr;
    used += (count * sizeof(T) + 255) / 256 * 256;
    return p;
  }
};

// Bounds of the sizes.  2^24 outputs and 2^27 rows or slots keep every count of tiles, and
// the offsets of one row, within 32 bits.
constexpr int64_t kMaxSlots = int64_t{1} << 27;
constexpr int kMaxOutputs = 1 << 24;
constexpr int64_t kMaxElements = int64_t{1} << 31;
constexpr int64_t kMaxBlocks = int64_t{1} << 22;   // of 512 threads: half of what one launch takes

// The layer's own shape and what these calls need besides.
int check_layer(int N, int K, int group_size, int bits) {
  if (int rc = check_shape(N, K, group_size)) return rc;
  if (K % 64 != 0) return fail(W4A16_ERR_UNSUPPORTED, "K=%d is not a multiple of 64", K);
  if (bits == 8 && N % 16 != 0) return fail(W4A16_ERR_UNSUPPORTED, "N=%d is not a multiple of 16 (8-bit weights)", N);
  if (N > kMaxOutputs) return fail(W4A16_ERR_UNSUPPORTED, "N=%d: at most %d outputs", N, kMaxOutputs);
  if (static_cast<int64_t>(N) * K * bits / 8 >= int64_t{1} << 32)
    return fail(W4A16_ERR_UNSUPPORTED, "N=%d K=%d: 2^32 bytes of codes or more", N, K);
  return W4A16_OK;
}

int log2_group(int g) { return g == 32 ? 5 : g == 64 ? 6 : g == 128 ? 7 : 30; }

Layers make_layers(const int32_t* qweight, const uint16_t* scales, const int32_t* qzeros, int group_size, int N, int K,
                   int bits, bool act) {
  Layers l;
  l.qw = reinterpret_cast<const uint32_t*>(qweight);
  l.scales = reinterpret_cast<const half_t*>(scales);
  l.zeros = qzeros ? Zeros{reinterpret_cast<const uint32_t*>(qzeros), 0} : Zeros{reinterpret_cast<const uint32_t*>(scales), 1};
  l.words = bits == 4 ? qweight_words(N, K, act) : qweight8_words(N, K, act);
  l.N = N;
  l.K = K;
  l.gshift = log2_group(group_size);
  l.G = K / group_size;
  return l;
}

// Row tiles that S slots of E experts can need.
int64_t most_tiles(int64_t S, int E, int height) { return S / height + (E < S ? E : S); }

SlotPlan take_plan(Carver& ws, int64_t S, int E, int64_t tiles, bool tile_of) {
  SlotPlan p;
  const int blocks = plan_blocks(S);
  p.sums = blocks > 1 ? ws.take<int32_t>(static_cast<size_t>(blocks + 2) * (E + 1)) : nullptr;
  p.tile_of = tile_of ? ws.take<int32_t>(S) : nullptr;
  p.counts = ws.take<int32_t>(2);
  p.order = ws.take<int32_t>(S);
  p.tiles = ws.take<RowTile>(tiles);
  return p;
}

// --- tile shapes ------------------------------------------------------------------------

// Compute units of a whole device.  A constant, so that the workspace functions need no device and
// agree with the calls; on fewer units the choices are slower ones, and no less right.
constexpr int kUnits = 256;

// A tile's place in a kernel: the height of the plan's full tiles; bm, the rows that the kernel's
// ring has room for (256: a workgroup per compute unit, 128: two, with half the memory each; 64:
// two of the 64-row kernel); its 64-column blocks, 4 or (bm 256) 1.
struct TileShape {
  int height, bm, nb;
};

// Time of a round of tiles against one of 256-row tiles of 256 columns: `full` with as many
// workgroups as run at once (tile_slots), `one` with at most one per compute unit.  Measured:
// whole calls of 64 experts of 256, 128 and 64 rows (N and K 4096, 4 bits), less 15 us (20 us) of
// launches: bm 256 570 / 378 / 276 us, 128 - / 343 / 250 us, 64 203 us for the last; back 564 /
// 401 / 298 us, 128 - / 362 / 262 us.  One per compute unit: eight experts of 256, 128, 64 rows
// 117 / 75 / 61 us, 64 45 us.  With half the memory alone on a compute unit 8-bit tiles wait for
// their shorter ring: 2588 rows against 2346 columns, K 2816 76 us, so 119 us.
struct TileCost {
  double one, full;
};

TileCost forward_cost(const TileShape& s, int rows) {
  constexpr double one[2][3] = {{0.73, 0.43, 0.33}, {0.33, 0.22, 0.15}};
  constexpr double full256[2][3] = {{1.0, 0.65, 0.47}, {0.40, 0.26, 0.20}};
  constexpr double full128[3] = {2.0, 1.18, 0.85};
  if (s.bm == 64) return {0.22, 0.68};
  const int n = s.nb == 1, i = rows == 256 ? 0 : rows == 128 ? 1 : 2;
  return s.bm == 256 ? TileCost{one[n][i], full256[n][i]} : TileCost{1.2 * one[0][i], full128[i]};
}

TileCost transposed_cost(const TileShape& s, int rows) {
  if (s.bm == 256) return rows == 256 ? TileCost{1.0, 1.0} : rows == 128 ? TileCost{0.60, 0.70} : TileCost{0.45, 0.51};
  return rows == 128 ? TileCost{0.75, 1.26} : TileCost{0.55, 0.89};
}

// Row tiles of S slots over E experts, their mean cost, and the largest with one per compute
// unit.  The groups' sizes are known on the device only: taken as 0.7 to 1.3 of the mean where
// there is more than one.
struct TileMix {
  double tiles = 0, one = 0, full = 0;
};

template <class Cost>
TileMix mix_of(int64_t S, int E, const TileShape& shape, Cost cost) {
  TileMix m;
  const int64_t used = E < S ? E : S;
  const double sizes[] = {1.0, 0.7, 0.85, 1.15, 1.3};
  const int count = used == 1 ? 1 : 5;
  for (int i = 0; i < count; ++i) {
    const int64_t rows = std::max<int64_t>(1, static_cast<int64_t>(static_cast<double>(S) / used * sizes[i] + 0.5));
    const auto add = [&](double n, int tile) {
      const TileCost c = cost(shape, tile);
      m.tiles += n, m.full += n * c.full;
      if (n > 0) m.one = std::max(m.one, c.one);
    };
    add(static_cast<double>(rows / shape.height), shape.height);
    const int rest = static_cast<int>(rows % shape.height);
    if (rest) add(1, rest_height(rest, shape.height));
  }
  m.full /= m.tiles;
  m.tiles *= static_cast<double>(used) / count;
  return m;
}

// Time of a product of S slots over E experts with `cols` output columns.  One expert's rounds
// are whole, of an estimated number of tiles half a round more on average.
double forward_time(int64_t S, int E, int cols, const TileShape& shape) {
  const TileMix m = mix_of(S, E, shape, forward_cost);
  const double wgs = m.tiles * ceil_div(cols, 64 * shape.nb);
  if (wgs <= kUnits) return m.one;
  const double rounds = wgs / (8 * tile_slots(shape.bm));
  return m.full * (rounds <= 1 ? 1.0 : E > 1 ? rounds + 0.5 : rounds < 8 ? std::ceil(rounds) : rounds);
}

// The shape of least time; narrow: 64-column tiles as well.
TileShape pick_forward(int64_t S, int E, int cols, bool narrow) {
  constexpr TileShape shapes[] = {{256, 256, 4}, {128, 256, 4}, {128, 128, 4}, {64, 64, 4},
                                  {256, 256, 1}, {128, 256, 1}, {64, 256, 1}};
  TileShape best = shapes[0];
  double least = 1e300;
  for (const TileShape& s : shapes) {
    if (s.nb == 1 && !narrow) continue;
    const double cost = forward_time(S, E, cols, s);
    if (cost < 0.999 * least) least = cost, best = s;
  }
  return best;
}

// Shape of the tiles and the most parts of a tile of the transposed product (see Pieces): parts
// of at least 512 outputs, partial sums of at most 512 MB.  The times here choose the shape
// alone; how many parts there are is the kernels' rule.
struct TransposedShape {
  int height, bm, most;
};

TransposedShape pick_transposed(int64_t S, int E, int outputs, int K) {
  constexpr TileShape shapes[] = {{256, 256, 4}, {128, 256, 4}, {64, 256, 4}, {128, 128, 4}, {64, 128, 4}};
  const int64_t fit = (int64_t{512} << 20) / (4 * S * K);
  TransposedShape best{256, 256, 1};
  best.most = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({int64_t{32}, fit, outputs / 512})));
  double least = 1e300;
  for (const TileShape& s : shapes) {
    const TileMix m = mix_of(S, E, s, transposed_cost);
    const int side = tile_slots(s.bm);
    const int64_t chunk = ceil_div(static_cast<int64_t>(m.tiles * ceil_div(K, 256) + 0.999), 8);
    const int64_t rest = chunk % side;
    double tail = rest == 0 ? 0 : rest <= 32 ? m.one : m.full;
    for (int f = 2; f <= best.most && f * rest <= 2 * side; ++f)
      tail = std::min(tail, (f * rest <= 32 ? m.one : m.full * ceil_div(rest * f, side)) / f +
                                f * (static_cast<float>(kPartCost) * rest / outputs));
    const double cost = static_cast<double>(chunk / side) * m.full + tail;
    if (cost < 0.999 * least) least = cost, best.height = s.height, best.bm = s.bm;
  }
  return best;
}

int64_t up8(int64_t n) { return (n + 7) / 8 * 8; }

// Allows a kernel its dynamic LDS; once per kernel and process (the value is static at the
// caller), on whichever device comes first: the runtime launches up to 160 KB without it as well.
hipError_t allow_lds(const void* kernel, size_t bytes) {
  return hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
}

int lds_status(hipError_t e) {
  if (e == hipSuccess) return W4A16_OK;
  return fail(W4A16_ERR_HIP, "hipFuncSetAttribute: %s", hipGetErrorString(e));
}

}  // namespace

// Launches that the entry points share (experts.hip).
// The slots of index grouped by expert; arguments as plan_slots_kernel.
void run_plan(const SlotPlan& p, const int32_t* index, int S, int E, int limit, int height, hipStream_t st);
// Act order: the valid slots' rows in stored channel order; the orders' inverses.
void run_gather(const SlotPlan& p, const half_t* x, const int32_t* index, const Layers& l, int S, int T, half_t* out,
                hipStream_t st);
void run_invert(const Layers& l, int E, int32_t* inverse, hipStream_t st);
// The transposed product over at most `tiles` row tiles; arguments as transposed_kernel.
int run_transposed(int bits, int bm, int64_t tiles, const half_t* a, int a_rows, int a_pitch, bool by_place,
                   const Layers& l, const SlotPlan& p, int slots, int n_begin, int n_end, int n_valid, int n_most, int most,
                   const TOut& to, hipStream_t st);

}  // namespace w4a16
