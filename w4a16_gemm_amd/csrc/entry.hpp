// Host-side helpers of the entry points of the mixtures of experts and of the vocabulary
// head: argument checks, workspace and launches.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>

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

SlotPlan take_plan(Carver& ws, int64_t S, int64_t tiles, bool tile_of) {
  SlotPlan p;
  p.tile_of = tile_of ? ws.take<int32_t>(S) : nullptr;
  p.counts = ws.take<int32_t>(2);
  p.order = ws.take<int32_t>(S);
  p.tiles = ws.take<RowTile>(tiles);
  return p;
}

// --- tile shapes ------------------------------------------------------------------------

constexpr int kUnits = 256;   // compute units

// Cost of a row tile against one of 256 rows: the weights are expanded for fewer rows.  (64
// experts of 256 / 128 / 64 rows, N and K 4096, 4 bits, whole calls: 549 / 366 / 268 us, back
// 564 / 401 / 298 us.)
double height_cost(int height) { return height == 256 ? 1.0 : height == 128 ? 0.64 : 0.45; }

// Row tiles of S slots over E experts, whose sizes are known on the device only: taken as
// equal, with half a tile more for each where there is more than one.
double tiles_of(int64_t S, int E, int height) {
  if (E == 1) return static_cast<double>(ceil_div(S, height));
  const double used = static_cast<double>(E < S ? E : S);
  const double per = static_cast<double>(S) / used / height;
  return used * (per <= 0.7 ? 1.0 : per + 0.5);
}

// Height of the full row tiles and the most parts of a tile of the transposed product (see
// Pieces): parts of at least 512 outputs, partial sums of at most 512 MB.
struct TransposedShape {
  int height, most;
};

TransposedShape pick_transposed(int64_t S, int E, int outputs, int K) {
  const int64_t fit = (int64_t{512} << 20) / (4 * S * K);
  TransposedShape best{256, 1};
  best.most = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({int64_t{16}, fit, outputs / 512})));
  double least = 1e300;
  for (int height : {256, 128, 64}) {
    const int64_t chunk = ceil_div(static_cast<int64_t>(tiles_of(S, E, height) * ceil_div(K, 256) + 0.999), 8);
    const int64_t rest = chunk % 32;
    double tail = rest ? 1.0 : 0.0;
    for (int f = 2; f <= best.most && f * rest <= 64; ++f) tail = std::min(tail, static_cast<double>(ceil_div(rest * f, 32)) / f + 0.02 * f);
    const double cost = (static_cast<double>(chunk / 32) + tail) * height_cost(height);
    if (cost < 0.999 * least) least = cost, best.height = height;
  }
  return best;
}

int64_t up8(int64_t n) { return (n + 7) / 8 * 8; }

// Allows a kernel its dynamic LDS; once per kernel and process (the value is static at the
// caller).
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
int run_transposed(int bits, int64_t tiles, const half_t* a, int a_rows, int a_pitch, bool by_place, const Layers& l,
                   const SlotPlan& p, int slots, int n_begin, int n_end, int n_valid, int n_most, int most, const TOut& to, hipStream_t st);

}  // namespace w4a16
