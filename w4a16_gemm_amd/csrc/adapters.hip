// Entry points of the low-rank adapters and the 8-bit activation checkpoints
// (w4a16_adapters.h): argument checks, kernel choice and launches.  Every launch is
// asynchronous on the caller's stream; the only scratch memory is the caller's workspace.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "internal.hpp"
#include "kernels/lora.hpp"
#include "w4a16_adapters.h"

namespace w4a16 {
namespace {

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

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
    if (b.ptr && !aligned(b.ptr, b.align))
      return fail(W4A16_ERR_MISALIGNED, "buffer %s is not %d-byte aligned", b.name, static_cast<int>(b.align));
  return W4A16_OK;
}

// Bounds on the sizes, which keep the launch grids below 2^32 threads but for those of the outer
// products and of the stream.  These, of 256 threads per workgroup, are checked by
// check_forward_shape and check_backward_shape: each may have half of what one launch takes.
// (No device holds the operands of a stream that is refused.)
constexpr int kMaxRows = 1 << 27;
constexpr int kMaxChannels = 1 << 24;
constexpr int64_t kMaxBlocks = int64_t{1} << 23;

int check_lora_shape(int M, int N, int K, int R, int L) {
  if (M <= 0 || N <= 0 || K <= 0) return fail(W4A16_ERR_INVALID_ARG, "sizes must be positive: M=%d N=%d K=%d", M, N, K);
  if (N % 8 != 0 || K % 8 != 0) return fail(W4A16_ERR_INVALID_ARG, "N=%d and K=%d must be multiples of 8", N, K);
  if (M > kMaxRows || N > kMaxChannels || K > kMaxChannels)
    return fail(W4A16_ERR_UNSUPPORTED, "M=%d N=%d K=%d: at most %d rows and %d channels", M, N, K, kMaxRows, kMaxChannels);
  if (R < 8 || R > 128 || R % 8 != 0) return fail(W4A16_ERR_UNSUPPORTED, "rank %d is not a multiple of 8 in 8..128", R);
  if (L < 1 || L > 65535) return fail(W4A16_ERR_UNSUPPORTED, "%d adapters, not 1..65535", L);
  return W4A16_OK;
}

int check_act_shape(int M, int K, int group_size) {
  if (M <= 0 || K <= 0) return fail(W4A16_ERR_INVALID_ARG, "sizes must be positive: M=%d K=%d", M, K);
  if (static_cast<int64_t>(M) * K >= int64_t{1} << 34)
    return fail(W4A16_ERR_UNSUPPORTED, "M=%d K=%d: at most 2^34 values per call", M, K);
  if (group_size != 32 && group_size != 64 && group_size != 128)
    return fail(W4A16_ERR_UNSUPPORTED, "group_size %d is not 32, 64 or 128", group_size);
  if (K % group_size != 0) return fail(W4A16_ERR_INVALID_ARG, "K=%d is not a multiple of group_size=%d", K, group_size);
  return W4A16_OK;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

int ceil_div(int a, int b) { return a / b + (a % b != 0); }

// --- workspace ----------------------------------------------------------------------

// Hands out 256-byte aligned pieces of the workspace; with base NULL it only adds them up,
// which is how the _workspace functions know the size.
struct Carver {
  unsigned char* base;
  size_t used = 0;
  template <typename T>
  T* take(size_t count) {
    T* p = base ? reinterpret_cast<T*>(base + used) : nullptr;
    used += up256(count * sizeof(T));
    return p;
  }
};

struct ByRow {
  half_t* frags;
  float* factors;
  uint16_t* wide;
};

struct ByRank {
  half_t* frags;
  float* units;
};

ByRow take_by_row(Carver& ws, int slots, int R) {
  half_t* f = ws.take<half_t>(static_cast<size_t>(slots) * 2 * row_frags(R) * 512);
  float* factors = ws.take<float>(static_cast<size_t>(slots) * kSlotRows);
  return {f, factors, ws.take<uint16_t>(static_cast<size_t>(slots) * 8)};
}

ByRank take_by_rank(Carver& ws, int slots, int R) {
  const size_t frags = static_cast<size_t>(slots) * ceil_div(R, 16);
  half_t* f = ws.take<half_t>(frags * 1024);
  return {f, ws.take<float>(frags * 16)};
}

SlotTable take_table(Carver& ws, int slots, int rows) {
  int2* meta = ws.take<int2>(slots);
  return {meta, ws.take<int32_t>(static_cast<size_t>(slots) * rows)};
}

// Memory of a row plan; without an index the rows need none.
RowPlan take_plan(Carver& ws, const int32_t* index, bool with_index, int M, int L) {
  RowPlan p{index, nullptr, nullptr, M, L};
  if (with_index) {
    p.off = ws.take<int32_t>(static_cast<size_t>(L) + 2);
    p.perm = ws.take<int32_t>(M);
  }
  return p;
}

void run_plan(const RowPlan& p, hipStream_t st) {
  if (p.index && p.off)
    hipLaunchKernelGGL(plan_rows_kernel, dim3(p.L + 1), dim3(1024), 0, st, p.index, p.M, p.L,
                       const_cast<int32_t*>(p.off), const_cast<int32_t*>(p.perm));
}

int tiles_of(const RowPlan& p, int T) { return tile_slots(p.M, p.L, p.index != nullptr, p.off != nullptr, T); }

int plan_slots(int M, int L, bool with_index) {
  return tile_slots(M, L, with_index, true, kSlotRows);
}

// The rules below take M / L for the rows per adapter, as if every one of the L adapters that are
// passed had the same part of the rows: the index lies on the device.  Results do not depend on it,
// times do where few of many adapters are used.  2048 rows, K = 4096, N = 14336, rank 16, all on one
// adapter, forward / backward with dx: of 1 adapter 35 / 45 us, of 8 36 / 59 us, of 64 36 / 94 us, and
// 16 adapters with nearly all rows on one 38 / 85 us; at rank 64 41 / 59, 41 / 74, 45 / 174 and 48 /
// 113 us; 4096 rows, K = N = 1536, rank 16: of 1 23 / 35 us, of 64 23 / 121 us.  (The gradients of 64
// adapters are 75 MB at rank 16 and 302 MB at rank 64 in the first shape, 15 and 60 us by
// themselves.)  A caller that knows which adapters a batch uses passes those alone.  Without an
// index the same figure is taken, so L = 1 is the call for one adapter.

// --- shrink -------------------------------------------------------------------------

// Rows per tile of a shrink, in 16s (wavefronts): 128 or 64 rows, once an adapter has that
// many on average; below that 16, with the wavefronts along the channels (512 rows x 11008 at
// rank 16: 6.4 us, in tiles of 64 rows 6.2).  With w transposed only the tiles of 64 rows and
// more, which take w through LDS.
int shrink_waves(int M, int L, int R, bool trans) {
  if (!trans && M / L < 64) return 1;
  return M / L >= 128 && (M > 512 || R > 32) ? 8 : 4;
}

// Slices of the long axis: a workgroup per compute unit (tiles of 16 rows: two), at least 256
// channels each (tiles of 16 rows: 512), and sums of the slices that stay small (8 MB) or an
// eighth of x (as much again when they are read).  A second workgroup on some compute units only makes the others wait (4096 rows
// x 28672 channels at rank 64: 50 us with 256, 52 us with 512; 2048 rows: 12 us with 256, 18 us
// with 128).  With an index an adapter's last tile is half full on average.  A power of two, so
// that a slice always falls to the same XCDs (8, in turn) and their L2 keeps its part of w (2048
// rows x 4096 of eight adapters at rank 64: 11.3 us in 8 slices, 13.8 us in 12).
int shrink_slices(int M, int L, int R, int C, bool with_index, bool trans, bool stream) {
  const int waves = stream ? shrink_waves(M, L, R, trans) : 1;
  const int tiles = ceil_div(M, 16 * waves) + (with_index ? L / 2 : 0);
  int want = waves == 1 ? ceil_div(512, ceil_div(M, 16)) : 256 / tiles;
  if (waves > 1) while (want & (want - 1)) want &= want - 1;
  const int64_t light = std::max<int64_t>(C / (16 * R), (int64_t{1} << 21) / (static_cast<int64_t>(M) * R));
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({want, C / (waves == 1 ? 512 : 256), M > 512 ? 16 : 32, light})));
}

template <bool TRANS>
void run_shrink(const half_t* x, const half_t* w, const RowPlan& plan, int C, int R, int S, float* out, SlotTable few,
                hipStream_t st) {
  const int waves = few.meta ? 1 : shrink_waves(plan.M, plan.L, R, TRANS);
  const dim3 grid(tiles_of(plan, 16 * waves) * S);
#define W4A16_SHRINK(NT_, D_) \
  do { \
    if (waves == 8) { \
      hipLaunchKernelGGL((lora_shrink_tall_kernel<NT_, 8, TRANS, (NT_ == 8 ? 2 : 4)>), grid, dim3(512), 0, st, x, w, plan, C, R, S, out); \
    } else if (waves == 4) { \
      hipLaunchKernelGGL((lora_shrink_tall_kernel<NT_, 4, TRANS, (NT_ == 8 ? 2 : 4)>), grid, dim3(256), 0, st, x, w, plan, C, R, S, out); \
    } else if constexpr (!TRANS) { \
      hipLaunchKernelGGL((lora_shrink_kernel<NT_, D_>), grid, dim3(256), 0, st, x, w, plan, C, R, S, out, few); \
    } \
  } while (0)
  const int nt = ceil_div(R, 16);
  if (nt == 1) W4A16_SHRINK(1, 4);
  else if (nt == 2) W4A16_SHRINK(2, 4);
  else if (nt <= 4) W4A16_SHRINK(4, 4);
  else W4A16_SHRINK(8, 2);
#undef W4A16_SHRINK
}

// --- expand -------------------------------------------------------------------------

void run_expand(const float* h, int S, const SlotTable& table, int slots, const half_t* w, const float* scaling, int L,
                const half_t* base, half_t* out, float* h_out, int C, int R, hipStream_t st) {
  const dim3 grid(slots, ceil_div(C, 512)), block(256);
#define W4A16_EXPAND(F_, P_) \
  hipLaunchKernelGGL((lora_expand_kernel<F_, P_>), grid, block, 0, st, h, S, table, w, scaling, L, base, out, h_out, C, R)
  if (R <= 16) W4A16_EXPAND(1, true);
  else if (R <= 32) W4A16_EXPAND(1, false);
  else if (R <= 64) W4A16_EXPAND(2, false);
  else if (R <= 96) W4A16_EXPAND(3, false);
  else W4A16_EXPAND(4, false);
#undef W4A16_EXPAND
}

// The whole forward in one launch where every workgroup (of one tile and 1024 output channels)
// can read its adapter's A again in the time of a launch, up to 96 KB of A, and all of them
// run at once.  Measured (graph replay, one launch against two): K = 1536, N = 1536, rank 16,
// one row 6.0 us against 7.4; K = 4096, N = 11008, rank 16, one row 9.1 against 7.9; K =
// 1536, N = 8960, rank 32, 256 rows of 32 adapters 30.5 against 19.2.
constexpr int kFusedA = 48 << 10;   // values

bool forward_fused(int M, int N, int K, int R, int L, bool with_index) {
  return M <= kInlineRows && R <= 64 && R * K <= kFusedA &&
         tile_slots(M, L, with_index, false, kFewRows) * ceil_div(N, 1024) <= 256;
}

void run_fused(const half_t* x, const half_t* a, const half_t* b, const float* scaling, const RowPlan& plan,
               const half_t* base, half_t* out, float* h_out, int K, int N, int R, hipStream_t st) {
  const dim3 grid(tiles_of(plan, 16) * ceil_div(N, 1024)), block(512);
#define W4A16_FUSED(F_, P_, D_) \
  hipLaunchKernelGGL((lora_fused_kernel<F_, P_, D_>), grid, block, 0, st, x, a, b, scaling, plan, base, out, h_out, K, N, R)
  if (R <= 16) W4A16_FUSED(1, true, 8);
  else if (R <= 32) W4A16_FUSED(1, false, 4);
  else W4A16_FUSED(2, false, 4);
#undef W4A16_FUSED
}

// `most` workgroups, 64 slots each at most.  Fewer of them read the weights less often, down
// to one round of two per compute unit in the forward pass (512; 2048 rows x 14336 in runs of
// eight adapters at rank 64: 30 us, with 1024 32 us, with 2048 37 us; 4096 x 28672 at rank 64:
// 96 us, 99 us with 1024, 120 us with 256).  dx runs beside the outer products, whose end it
// has to fill: 1024 (2500 rows of four adapters, K = N = 4096, rank 64: 25 us, with 512 29 us).
constexpr int kForwardBlocks = 512, kBackwardBlocks = 1024;

int stream_group(int C, int slots, int most) {
  const int64_t all = static_cast<int64_t>(slots) * ceil_div(C, 512);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(64, (all + most - 1) / most)));
}

int64_t stream_blocks(int C, int slots, int group) {
  return static_cast<int64_t>(ceil_div(C, 512)) * ceil_div(slots, group);
}

StreamArgs stream_args(const ByRow& f, const float* h, const float* scaling, const SlotTable& table, const half_t* w,
                       const half_t* base, half_t* out, int C, int R, int L, int slots, int most) {
  return {f.frags, f.factors, f.wide, h, scaling, table, w, base, out, C, R, L, slots, stream_group(C, slots, most)};
}

int stream_blocks(const StreamArgs& s) { return static_cast<int>(stream_blocks(s.C, s.slots, s.group)); }

template <bool TRANS, bool BASE>
void run_stream(const StreamArgs& s, hipStream_t st) {
  const dim3 grid(stream_blocks(s)), block(256);
#define W4A16_STREAM(F_, P_, D_) \
  hipLaunchKernelGGL((lora_stream_kernel<F_, P_, TRANS, BASE, D_>), grid, block, 0, st, s)
  if constexpr (!TRANS) {   // ranks up to 64 of the backward pass are in the products kernel
    if (s.R <= 64) {
      if (s.R <= 16) W4A16_STREAM(1, true, 2);
      else if (s.R <= 32) W4A16_STREAM(1, false, 2);
      else W4A16_STREAM(2, false, 2);
      return;
    }
  }
  if (s.R <= 96) W4A16_STREAM(3, false, 2);
  else W4A16_STREAM(4, false, 2);
#undef W4A16_STREAM
}

// --- outer --------------------------------------------------------------------------

// The vectors of the outer products: binary16 rows, or a checkpoint.
struct Kept {
  const half_t* x;
  const uint8_t* codes;
  const half_t* scales;
  int gshift;
};

// Workgroups that share the rows of 128 channels, `groups` of them being there with one
// each: up to one per compute unit, as long as each keeps 32 slots of an average adapter.
int outer_parts(int M, int L, int64_t groups) {
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({256 / groups, M / L / (32 * kSlotRows), 16})));
}

// Ranks per block of an outer product, in 16s.  Blocks of 32 ranks read x or dy again, from
// the L2 of their XCD, for every further block; blocks of 64 leave registers for one wavefront
// per SIMD, and were slower for every size (4096 rows, K = 8192, N = 28672, rank 64, with dx:
// 103 us in one launch in blocks of 32, 117 us in blocks of 64 and two launches).
int outer_nt(int R) { return R <= 16 ? 1 : 2; }

int64_t outer_groups(int C, int R, int L, int row_waves) {
  const int ranks = ceil_div(R, 16 * outer_nt(R));   // more than one: whole eights of blocks of channels
  const int width = 512 / row_waves;
  return static_cast<int64_t>(ranks == 1 ? ceil_div(C, width) : ceil_div(C, 8 * width) * 8 * ranks) * L;
}

// Wavefronts of a workgroup (of 4) that share the rows of 128 channels.  With few rows per
// adapter and more workgroups than fit at once, each wavefront takes channels of its own and
// all the rows: a quarter of the workgroups, and no sums to add (700 rows of 12 adapters, K =
// N = 4096, rank 40: 27 -> 15 us; 1024 rows of 16, rank 16: 19 -> 13 us; but 1111 rows of 6, K =
// 1536, N = 8960, rank 32: 14 -> 19 us).
int outer_row_waves(int M, int N, int K, int R, int L) {
  return M / L <= 128 && outer_groups(K, R, L, 4) + outer_groups(N, R, L, 4) >= 768 ? 1 : 4;
}

// dB, dA and dx go out in one launch up to rank 64.  Above, the registers for the weights of dx
// would hold the outer products back (300 rows, rank 128: 27 us in one launch, 24 us in two).
bool products_together(int R) { return R <= 64; }

OuterArgs outer_args(const Kept& k, const ByRank& f, const float* h, const float* scaling, const RowPlan& plan,
                     float* grad, int C, int R, int parts, int row_waves) {
  return {k.x, k.codes, k.scales, k.gshift, f.frags, f.units, h, scaling, plan, grad, C, R, parts, row_waves};
}

int outer_blocks(const OuterArgs& o) { return static_cast<int>(outer_groups(o.C, o.R, o.plan.L, o.row_waves) * o.parts); }

template <bool Q8>
void run_outers(const OuterArgs& b, const OuterArgs& a, hipStream_t st) {
  const int nb = outer_blocks(b), na = outer_blocks(a);
  hipLaunchKernelGGL((lora_outers_kernel<Q8>), dim3(nb + na), dim3(256), 0, st, b, nb, a);
}

template <int NT, int F, bool Q8>
void run_products(const OuterArgs& b, const OuterArgs& a, const StreamArgs& dx, hipStream_t st) {
  const int nb = outer_blocks(b), na = outer_blocks(a);
  const dim3 grid(nb + na + (dx.out ? stream_blocks(dx) : 0)), block(256);
  if (!dx.out) hipLaunchKernelGGL((lora_products_kernel<NT, F, Q8, false, false>), grid, block, 0, st, b, nb, a, na, dx);
  else if (!dx.base) hipLaunchKernelGGL((lora_products_kernel<NT, F, Q8, true, false>), grid, block, 0, st, b, nb, a, na, dx);
  else hipLaunchKernelGGL((lora_products_kernel<NT, F, Q8, true, true>), grid, block, 0, st, b, nb, a, na, dx);
}

// --- sizes --------------------------------------------------------------------------

int check_stream(int M, int L, bool with_index, int C, int most) {
  const int slots = plan_slots(M, L, with_index);
  if (stream_blocks(C, slots, stream_group(C, slots, most)) > kMaxBlocks)
    return fail(W4A16_ERR_UNSUPPORTED, "M=%d rows of %d adapters over %d channels are too many for one call", M, L, C);
  return W4A16_OK;
}

int check_forward_shape(int M, int N, int K, int R, int L, bool with_index) {
  if (int rc = check_lora_shape(M, N, K, R, L)) return rc;
  return M > kInlineRows ? check_stream(M, L, with_index, N, kForwardBlocks) : W4A16_OK;
}

int check_backward_shape(int M, int N, int K, int R, int L, bool with_index) {
  if (int rc = check_lora_shape(M, N, K, R, L)) return rc;
  if (outer_groups(N, R, L, 4) + outer_groups(K, R, L, 4) >= kMaxBlocks)
    return fail(W4A16_ERR_UNSUPPORTED, "gradients of %d adapters for N=%d, K=%d are too large for one call", L, N, K);
  return check_stream(M, L, with_index, K, kBackwardBlocks);
}

// --- forward ------------------------------------------------------------------------

struct ForwardMemory {
  RowPlan plan;
  float* part;       // [S][M][R], or [slots][S][16][R] for few rows
  int S, slots;
  bool fused, stream;
  ByRow h;
  float* h_far;      // [M][R]: h of the slots that are not whole, where the caller does not want it
  SlotTable table;
};

ForwardMemory forward_memory(Carver& ws, const int32_t* index, bool with_index, int M, int N, int K, int R,
                             int L) {
  ForwardMemory m{};
  m.fused = forward_fused(M, N, K, R, L, with_index);
  if (m.fused) {
    m.plan = RowPlan{index, nullptr, nullptr, M, L};
    return m;
  }
  m.stream = M > kInlineRows;
  m.plan = take_plan(ws, index, with_index && m.stream, M, L);
  m.S = shrink_slices(M, L, R, K, with_index, false, m.stream);
  if (m.stream) {
    m.slots = plan_slots(M, L, with_index);
    m.part = ws.take<float>(static_cast<size_t>(m.S) * M * R);
    m.h = take_by_row(ws, m.slots, R);
    m.h_far = ws.take<float>(static_cast<size_t>(M) * R);
    m.table = take_table(ws, m.slots, kSlotRows);
  } else {
    m.slots = tile_slots(M, L, with_index, false, kFewRows);
    m.part = ws.take<float>(static_cast<size_t>(m.slots) * m.S * kFewRows * R);
    m.table = take_table(ws, m.slots, kFewRows);
  }
  return m;
}

// --- backward -----------------------------------------------------------------------

struct BackwardMemory {
  RowPlan plan;
  float* part;       // g: [S][M][R]
  int S, slots;
  ByRank h, g;
  float* g_far;      // [M][R]: g of the slots that are not whole
  ByRow g_rows;
  SlotTable table;
  int parts, row_waves;   // of the outer products
  float *da, *db;    // [parts][L][R][K], [parts][L][N][R], where there is more than one part
};

BackwardMemory backward_memory(Carver& ws, const int32_t* index, bool with_index, int M, int N, int K, int R,
                               int L) {
  BackwardMemory m{};
  m.plan = take_plan(ws, index, with_index, M, L);
  m.S = shrink_slices(M, L, R, N, with_index, true, true);
  m.part = ws.take<float>(static_cast<size_t>(m.S) * M * R);
  m.slots = plan_slots(M, L, with_index);
  m.h = take_by_rank(ws, m.slots, R);
  m.g = take_by_rank(ws, m.slots, R);
  m.g_far = ws.take<float>(static_cast<size_t>(M) * R);
  m.g_rows = take_by_row(ws, m.slots, R);
  m.table = take_table(ws, m.slots, kSlotRows);
  m.row_waves = outer_row_waves(M, N, K, R, L);
  m.parts = outer_parts(M, L, outer_groups(K, R, L, m.row_waves) + outer_groups(N, R, L, m.row_waves));
  if (m.parts > 1) {
    m.da = ws.take<float>(static_cast<size_t>(m.parts) * L * R * K);
    m.db = ws.take<float>(static_cast<size_t>(m.parts) * L * N * R);
  }
  return m;
}

int check_workspace(const void* ws, size_t have, size_t need) {
  if (need > 0 && !ws) return fail(W4A16_ERR_INVALID_ARG, "NULL workspace, this call needs %zu bytes", need);
  if (have >= need) return W4A16_OK;
  return fail(W4A16_ERR_INVALID_ARG, "workspace of %zu bytes, this call needs %zu", have, need);
}

struct BackwardArgs {
  const uint16_t *dy, *a, *b;
  const float* h;
  const int32_t* index;
  const float* scaling;
  const uint16_t* dx0;
  int M, N, K, R, L;
  uint16_t* dx;
  float *da, *db;
  void* workspace;
  size_t workspace_bytes;
  void* stream;
};

template <bool Q8>
int run_backward(const BackwardArgs& c, const Kept& kept) {
  const Buffer bufs[] = {{c.dy, 16, true, "dy"},       {c.a, 16, true, "a"},     {c.b, 16, true, "b"},
                         {c.h, 16, true, "h"},         {c.da, 16, true, "da"},   {c.db, 16, true, "db"},
                         {c.dx0, 16, false, "dx0"},    {c.dx, 16, false, "dx"},  {c.index, 4, false, "index"},
                         {c.scaling, 4, false, "scaling"}, {c.workspace, 16, false, "workspace"}};
  if (int rc = check_buffers(bufs)) return rc;
  if (c.dx0 && !c.dx) return fail(W4A16_ERR_INVALID_ARG, "dx0 is given without dx");
  Carver size{nullptr}, ws{static_cast<unsigned char*>(c.workspace)};
  backward_memory(size, nullptr, c.index != nullptr, c.M, c.N, c.K, c.R, c.L);
  if (int rc = check_workspace(c.workspace, c.workspace_bytes, size.used)) return rc;
  const BackwardMemory m = backward_memory(ws, c.index, c.index != nullptr, c.M, c.N, c.K, c.R, c.L);
  const auto st = static_cast<hipStream_t>(c.stream);
  const auto* dy = reinterpret_cast<const half_t*>(c.dy);
  run_plan(m.plan, st);
  run_shrink<true>(dy, reinterpret_cast<const half_t*>(c.b), m.plan, c.N, c.R, m.S, m.part, SlotTable{}, st);
  const SplitTask th{c.h, 1, m.h.frags, m.h.units, nullptr, nullptr, nullptr, nullptr, nullptr};
  const SplitTask tg{m.part, m.S, m.g.frags, m.g.units, c.dx ? m.g_rows.frags : nullptr, m.g_rows.factors,
                     m.g_rows.wide, nullptr, m.g_far};
  hipLaunchKernelGGL(lora_split_kernel, dim3(m.slots, 2), dim3(512), 0, st, th, tg, c.scaling, m.table, m.plan, c.R);
  const bool whole = m.parts == 1;
  const OuterArgs ob = outer_args(Kept{dy, nullptr, nullptr, 0}, m.h, c.h, c.scaling, m.plan, whole ? c.db : m.db, c.N,
                                  c.R, m.parts, m.row_waves);
  const OuterArgs oa = outer_args(kept, m.g, m.g_far, c.scaling, m.plan, whole ? c.da : m.da, c.K, c.R, m.parts,
                                  m.row_waves);
  const StreamArgs dx = stream_args(m.g_rows, m.g_far, c.scaling, m.table, reinterpret_cast<const half_t*>(c.a),
                                    reinterpret_cast<const half_t*>(c.dx0), reinterpret_cast<half_t*>(c.dx), c.K, c.R, c.L,
                                    m.slots, kBackwardBlocks);
  if (products_together(c.R)) {
    if (c.R <= 16) run_products<1, 1, Q8>(ob, oa, dx, st);
    else if (c.R <= 32) run_products<2, 1, Q8>(ob, oa, dx, st);
    else run_products<2, 2, Q8>(ob, oa, dx, st);
  } else {
    run_outers<Q8>(ob, oa, st);
    if (dx.out) dx.base ? run_stream<true, true>(dx, st) : run_stream<true, false>(dx, st);
  }
  if (!whole) {
    auto task = [&](const float* parts, float* out, size_t count) {
      return PartsTask{reinterpret_cast<const float4_t*>(parts), reinterpret_cast<float4_t*>(out), count / 4, m.parts};
    };
    const PartsTask ta = task(m.da, c.da, static_cast<size_t>(c.L) * c.R * c.K);
    const PartsTask tb = task(m.db, c.db, static_cast<size_t>(c.L) * c.N * c.R);
    const size_t most = std::max(ta.quads, tb.quads);
    hipLaunchKernelGGL(lora_sum_parts_kernel, dim3(static_cast<unsigned>((most + 255) / 256), 2), dim3(256), 0, st, ta, tb);
  }
  return check_launch("lora backward launch");
}

}  // namespace
}  // namespace w4a16

using namespace w4a16;

extern "C" size_t w4a16_lora_forward_workspace(int M, int N, int K, int R, int L, int with_index) {
  if (check_forward_shape(M, N, K, R, L, with_index != 0) != W4A16_OK) return 0;
  Carver size{nullptr};
  forward_memory(size, nullptr, with_index != 0, M, N, K, R, L);
  return size.used;
}

extern "C" int w4a16_lora_forward(const uint16_t* y, const uint16_t* x, const uint16_t* a, const uint16_t* b,
                                  const int32_t* index, const float* scaling, int M, int N, int K, int R, int L,
                                  uint16_t* out, float* h, void* workspace, size_t workspace_bytes, void* stream) {
  begin_call();
  if (int rc = check_forward_shape(M, N, K, R, L, index != nullptr)) return rc;
  const Buffer bufs[] = {{y, 16, true, "y"},           {x, 16, true, "x"},          {a, 16, true, "a"},
                         {b, 16, true, "b"},           {out, 16, true, "out"},      {h, 16, false, "h"},
                         {index, 4, false, "index"},   {scaling, 4, false, "scaling"},
                         {workspace, 16, false, "workspace"}};
  if (int rc = check_buffers(bufs)) return rc;
  Carver size{nullptr}, ws{static_cast<unsigned char*>(workspace)};
  forward_memory(size, nullptr, index != nullptr, M, N, K, R, L);
  if (int rc = check_workspace(workspace, workspace_bytes, size.used)) return rc;
  const ForwardMemory m = forward_memory(ws, index, index != nullptr, M, N, K, R, L);
  const auto st = static_cast<hipStream_t>(stream);
  const auto* yh = reinterpret_cast<const half_t*>(y);
  const auto* bh = reinterpret_cast<const half_t*>(b);
  auto* oh = reinterpret_cast<half_t*>(out);
  const auto* xh = reinterpret_cast<const half_t*>(x);
  const auto* ah = reinterpret_cast<const half_t*>(a);
  if (m.fused) {
    run_fused(xh, ah, bh, scaling, m.plan, yh, oh, h, K, N, R, st);
    return check_launch("lora forward launch");
  }
  run_plan(m.plan, st);
  run_shrink<false>(xh, ah, m.plan, K, R, m.S, m.part, m.stream ? SlotTable{} : m.table, st);
  if (m.stream) {
    const SplitTask t{m.part, m.S, nullptr, nullptr, m.h.frags, m.h.factors, m.h.wide, h, h ? nullptr : m.h_far};
    hipLaunchKernelGGL(lora_split_kernel, dim3(m.slots, 1), dim3(512), 0, st, t, t, scaling, m.table, m.plan, R);
    run_stream<false, true>(stream_args(m.h, h ? h : m.h_far, scaling, m.table, bh, yh, oh, N, R, L, m.slots, kForwardBlocks), st);
  } else {
    run_expand(m.part, m.S, m.table, m.slots, bh, scaling, L, yh, oh, h, N, R, st);
  }
  return check_launch("lora forward launch");
}

extern "C" size_t w4a16_lora_backward_workspace(int M, int N, int K, int R, int L, int with_index) {
  if (check_backward_shape(M, N, K, R, L, with_index != 0) != W4A16_OK) return 0;
  Carver size{nullptr};
  backward_memory(size, nullptr, with_index != 0, M, N, K, R, L);
  return size.used;
}

extern "C" int w4a16_lora_backward(const uint16_t* dy, const uint16_t* x, const uint16_t* a, const uint16_t* b,
                                   const float* h, const int32_t* index, const float* scaling, const uint16_t* dx0,
                                   int M, int N, int K, int R, int L, uint16_t* dx, float* da, float* db,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  begin_call();
  if (int rc = check_backward_shape(M, N, K, R, L, index != nullptr)) return rc;
  const Buffer bufs[] = {{x, 16, true, "x"}};
  if (int rc = check_buffers(bufs)) return rc;
  return run_backward<false>(
      BackwardArgs{dy, a, b, h, index, scaling, dx0, M, N, K, R, L, dx, da, db, workspace, workspace_bytes, stream},
      Kept{reinterpret_cast<const half_t*>(x), nullptr, nullptr, 0});
}

extern "C" int w4a16_lora_backward_q8(const uint16_t* dy, const uint8_t* codes, const uint16_t* scales, int group_size,
                                      const uint16_t* a, const uint16_t* b, const float* h, const int32_t* index,
                                      const float* scaling, const uint16_t* dx0, int M, int N, int K, int R, int L,
                                      uint16_t* dx, float* da, float* db, void* workspace, size_t workspace_bytes,
                                      void* stream) {
  begin_call();
  if (int rc = check_backward_shape(M, N, K, R, L, index != nullptr)) return rc;
  if (int rc = check_act_shape(M, K, group_size)) return rc;
  const Buffer bufs[] = {{codes, 8, true, "codes"}, {scales, 2, true, "scales"}};
  if (int rc = check_buffers(bufs)) return rc;
  return run_backward<true>(
      BackwardArgs{dy, a, b, h, index, scaling, dx0, M, N, K, R, L, dx, da, db, workspace, workspace_bytes, stream},
      Kept{nullptr, codes, reinterpret_cast<const half_t*>(scales), group_size == 32 ? 5 : group_size == 64 ? 6 : 7});
}

extern "C" int w4a16_act_quantize(const uint16_t* x, int M, int K, int group_size, uint8_t* codes, uint16_t* scales,
                                  void* stream) {
  begin_call();
  if (int rc = check_act_shape(M, K, group_size)) return rc;
  const Buffer bufs[] = {{x, 16, true, "x"}, {codes, 8, true, "codes"}, {scales, 2, true, "scales"}};
  if (int rc = check_buffers(bufs)) return rc;
  const size_t chunks = static_cast<size_t>(M) * (K / 8);
  const dim3 grid(static_cast<unsigned>((chunks + 256 * kActRuns - 1) / (256 * kActRuns))), block(256);
  const auto st = static_cast<hipStream_t>(stream);
  const auto* xh = reinterpret_cast<const half_t*>(x);
  auto* sh = reinterpret_cast<half_t*>(scales);
  if (group_size == 32) hipLaunchKernelGGL((act_quantize_kernel<4>), grid, block, 0, st, xh, codes, sh, chunks);
  else if (group_size == 64) hipLaunchKernelGGL((act_quantize_kernel<8>), grid, block, 0, st, xh, codes, sh, chunks);
  else hipLaunchKernelGGL((act_quantize_kernel<16>), grid, block, 0, st, xh, codes, sh, chunks);
  return check_launch("act quantize launch");
}

extern "C" int w4a16_act_dequantize(const uint8_t* codes, const uint16_t* scales, int M, int K, int group_size,
                                    uint16_t* x, void* stream) {
  begin_call();
  if (int rc = check_act_shape(M, K, group_size)) return rc;
  const Buffer bufs[] = {{codes, 8, true, "codes"}, {scales, 2, true, "scales"}, {x, 16, true, "x"}};
  if (int rc = check_buffers(bufs)) return rc;
  const size_t chunks = static_cast<size_t>(M) * (K / 8);
  hipLaunchKernelGGL(act_dequantize_kernel, dim3(static_cast<unsigned>((chunks + 255) / 256)), dim3(256), 0,
                     static_cast<hipStream_t>(stream), codes, reinterpret_cast<const half_t*>(scales),
                     reinterpret_cast<half_t*>(x), chunks, group_size == 32 ? 2 : group_size == 64 ? 3 : 4);
  return check_launch("act dequantize launch");
}
