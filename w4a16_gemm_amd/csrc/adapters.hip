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

// Bounds of the launch grids (their sizes in threads stay below 2^32).
constexpr int kMaxRows = 1 << 27;
constexpr int kMaxChannels = 1 << 24;

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

// --- row plan -----------------------------------------------------------------------

size_t plan_bytes(int M, int L) { return up256((static_cast<size_t>(L) + 2 + M) * sizeof(int32_t)); }

// A plan in memory, taken from the front of the workspace.
RowPlan make_plan(const int32_t* index, int M, int L, unsigned char*& ws, hipStream_t st) {
  RowPlan p{index, nullptr, nullptr, M, L};
  auto* off = reinterpret_cast<int32_t*>(ws);
  int32_t* perm = off + L + 2;
  ws += plan_bytes(M, L);
  hipLaunchKernelGGL(plan_rows_kernel, dim3(L + 1), dim3(1024), 0, st, index, M, L, off, perm);
  p.off = off;
  p.perm = perm;
  return p;
}

// --- shrink -------------------------------------------------------------------------

// Slices of the long axis: enough workgroups to fill the GPU at few rows, at least 512
// channels (16 steps) per slice.
int shrink_slices(int M, int C) {
  const int tiles = ceil_div(M, 16);
  const int want = std::max(1, 256 / tiles);
  return std::max(1, std::min({want, C / 512, 16}));
}

size_t part_bytes(int S, int M, int R) { return up256(sizeof(float) * S * M * R); }

void run_shrink(const half_t* x, const half_t* w, const RowPlan& plan, int C, int R, int S, float* out, hipStream_t st) {
  const dim3 grid(tile_slots(plan, 16), S), block(256);
  switch ((R + 15) / 16) {
#define W4A16_SHRINK(NT_) \
    case NT_: hipLaunchKernelGGL((lora_shrink_kernel<NT_, 1, 4>), grid, block, 0, st, x, w, plan, C, R, out); break;
    W4A16_SHRINK(1) W4A16_SHRINK(2) W4A16_SHRINK(3) W4A16_SHRINK(4)
    W4A16_SHRINK(5) W4A16_SHRINK(6) W4A16_SHRINK(7) W4A16_SHRINK(8)
#undef W4A16_SHRINK
  }
}

// --- expand -------------------------------------------------------------------------

template <bool TRANS>
void run_expand(const float* h, int S, const half_t* w, const float* scaling, const RowPlan& plan, const half_t* base,
                half_t* out, float* h_out, int C, int R, hipStream_t st) {
  const bool wide = plan.M / plan.L >= 64;
  const dim3 grid(tile_slots(plan, wide ? 64 : 16), ceil_div(C, 512)), block(256);
#define W4A16_EXPAND(F_, P_) \
  do { \
    if (wide) hipLaunchKernelGGL((lora_expand_kernel<F_, P_, 4, TRANS>), grid, block, 0, st, h, S, w, scaling, plan, \
                                 base, out, h_out, C, R); \
    else hipLaunchKernelGGL((lora_expand_kernel<F_, P_, 1, TRANS>), grid, block, 0, st, h, S, w, scaling, plan, base, \
                            out, h_out, C, R); \
  } while (0)
  if (R <= 16) W4A16_EXPAND(1, true);
  else if (R <= 32) W4A16_EXPAND(1, false);
  else if (R <= 64) W4A16_EXPAND(2, false);
  else if (R <= 96) W4A16_EXPAND(3, false);
  else W4A16_EXPAND(4, false);
#undef W4A16_EXPAND
}

// --- outer --------------------------------------------------------------------------

// The vectors of the outer products: binary16 rows, or a checkpoint.
struct Kept {
  const half_t* x;
  const uint8_t* codes;
  const half_t* scales;
  int gshift;
};

struct Frags {
  half_t* frags;
  int32_t* exps;
};

size_t frag_bytes(int slots, int R) {
  return up256(static_cast<size_t>(slots) * ceil_div(R, 16) * 2048) + up256(static_cast<size_t>(slots) * sizeof(int32_t));
}

Frags take_frags(int slots, int R, unsigned char*& ws) {
  Frags f{reinterpret_cast<half_t*>(ws),
          reinterpret_cast<int32_t*>(ws + up256(static_cast<size_t>(slots) * ceil_div(R, 16) * 2048))};
  ws += frag_bytes(slots, R);
  return f;
}

template <bool Q8, bool CMAJOR>
void run_outer(const Kept& k, const Frags& f, const float* scaling, const RowPlan& plan, float* grad, int C, int R,
               hipStream_t st) {
#define W4A16_OUTER(NT_, W_, D_) \
  hipLaunchKernelGGL((lora_outer_kernel<NT_, W_, D_, Q8, CMAJOR>), dim3(ceil_div(C, 128), ceil_div(R, 16 * NT_), plan.L), \
                     dim3(64 * W_), 0, st, k.x, k.codes, k.scales, k.gshift, f.frags, f.exps, scaling, plan, grad, C, R)
  if (R <= 16) W4A16_OUTER(1, 8, 3);
  else if (R <= 32) W4A16_OUTER(2, 8, 2);
  else W4A16_OUTER(4, 4, 2);
#undef W4A16_OUTER
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

int backward_slots(int M, int L, bool with_index) {
  return with_index ? M / kSlotRows + L + 1 : ceil_div(M, kSlotRows);
}

size_t backward_bytes(int M, int N, int K, int R, int L, bool with_index) {
  (void)K;
  return (with_index ? plan_bytes(M, L) : 0) + up256(sizeof(half_t) * L * R * N) +
         part_bytes(shrink_slices(M, N), M, R) + 2 * frag_bytes(backward_slots(M, L, with_index), R);
}

template <bool Q8>
int run_backward(const BackwardArgs& c, const Kept& kept) {
  const Buffer bufs[] = {{c.dy, 16, true, "dy"},       {c.a, 16, true, "a"},     {c.b, 16, true, "b"},
                         {c.h, 16, true, "h"},         {c.da, 16, true, "da"},   {c.db, 16, true, "db"},
                         {c.dx0, 16, false, "dx0"},    {c.dx, 16, false, "dx"},  {c.index, 4, false, "index"},
                         {c.scaling, 4, false, "scaling"}, {c.workspace, 16, true, "workspace"}};
  if (int rc = check_buffers(bufs)) return rc;
  if (c.dx0 && !c.dx) return fail(W4A16_ERR_INVALID_ARG, "dx0 is given without dx");
  const size_t need = backward_bytes(c.M, c.N, c.K, c.R, c.L, c.index != nullptr);
  if (c.workspace_bytes < need)
    return fail(W4A16_ERR_INVALID_ARG, "workspace of %zu bytes, this call needs %zu", c.workspace_bytes, need);
  const auto st = static_cast<hipStream_t>(c.stream);
  auto* ws = static_cast<unsigned char*>(c.workspace);
  RowPlan plan{nullptr, nullptr, nullptr, c.M, c.L};
  if (c.index) plan = make_plan(c.index, c.M, c.L, ws, st);
  auto* bt = reinterpret_cast<half_t*>(ws);
  ws += up256(sizeof(half_t) * c.L * c.R * c.N);
  auto* g = reinterpret_cast<float*>(ws);
  const int S = shrink_slices(c.M, c.N);
  ws += part_bytes(S, c.M, c.R);
  const int slots = backward_slots(c.M, c.L, c.index != nullptr);
  const Frags fh = take_frags(slots, c.R, ws), fg = take_frags(slots, c.R, ws);
  const auto* dy = reinterpret_cast<const half_t*>(c.dy);
  const auto* a = reinterpret_cast<const half_t*>(c.a);
  const auto* b = reinterpret_cast<const half_t*>(c.b);
  hipLaunchKernelGGL(lora_transpose_kernel, dim3(ceil_div(c.N, kTransposeRows), c.L), dim3(256),
                     sizeof(half_t) * kTransposeRows * (c.R + 2), st, b, bt, c.N, c.R);
  run_shrink(dy, bt, plan, c.N, c.R, S, g, st);
  hipLaunchKernelGGL(lora_split_kernel, dim3(slots, 2), dim3(256), 0, st, SplitTask{c.h, 1, fh.frags, fh.exps},
                     SplitTask{g, S, fg.frags, fg.exps}, plan, c.R);
  run_outer<false, true>(Kept{dy, nullptr, nullptr, 0}, fh, c.scaling, plan, c.db, c.N, c.R, st);
  run_outer<Q8, false>(kept, fg, c.scaling, plan, c.da, c.K, c.R, st);
  if (c.dx)
    run_expand<true>(g, S, a, c.scaling, plan, reinterpret_cast<const half_t*>(c.dx0), reinterpret_cast<half_t*>(c.dx),
                     nullptr, c.K, c.R, st);
  return check_launch("lora backward launch");
}

}  // namespace
}  // namespace w4a16

using namespace w4a16;

extern "C" size_t w4a16_lora_forward_workspace(int M, int N, int K, int R, int L, int with_index) {
  if (check_lora_shape(M, N, K, R, L) != W4A16_OK) return 0;
  return (with_index && M > kInlineRows ? plan_bytes(M, L) : 0) + part_bytes(shrink_slices(M, K), M, R);
}

extern "C" int w4a16_lora_forward(const uint16_t* y, const uint16_t* x, const uint16_t* a, const uint16_t* b,
                                  const int32_t* index, const float* scaling, int M, int N, int K, int R, int L,
                                  uint16_t* out, float* h, void* workspace, size_t workspace_bytes, void* stream) {
  begin_call();
  if (int rc = check_lora_shape(M, N, K, R, L)) return rc;
  const Buffer bufs[] = {{y, 16, true, "y"},           {x, 16, true, "x"},          {a, 16, true, "a"},
                         {b, 16, true, "b"},           {out, 16, true, "out"},      {h, 16, false, "h"},
                         {index, 4, false, "index"},   {scaling, 4, false, "scaling"},
                         {workspace, 16, true, "workspace"}};
  if (int rc = check_buffers(bufs)) return rc;
  const size_t need = w4a16_lora_forward_workspace(M, N, K, R, L, index != nullptr);
  if (workspace_bytes < need)
    return fail(W4A16_ERR_INVALID_ARG, "workspace of %zu bytes, this call needs %zu", workspace_bytes, need);
  const auto st = static_cast<hipStream_t>(stream);
  auto* ws = static_cast<unsigned char*>(workspace);
  RowPlan plan{index, nullptr, nullptr, M, L};
  if (index && M > kInlineRows) plan = make_plan(index, M, L, ws, st);
  auto* part = reinterpret_cast<float*>(ws);
  const int S = shrink_slices(M, K);
  run_shrink(reinterpret_cast<const half_t*>(x), reinterpret_cast<const half_t*>(a), plan, K, R, S, part, st);
  run_expand<false>(part, S, reinterpret_cast<const half_t*>(b), scaling, plan, reinterpret_cast<const half_t*>(y),
                    reinterpret_cast<half_t*>(out), h, N, R, st);
  return check_launch("lora forward launch");
}

extern "C" size_t w4a16_lora_backward_workspace(int M, int N, int K, int R, int L, int with_index) {
  if (check_lora_shape(M, N, K, R, L) != W4A16_OK) return 0;
  return backward_bytes(M, N, K, R, L, with_index != 0);
}

extern "C" int w4a16_lora_backward(const uint16_t* dy, const uint16_t* x, const uint16_t* a, const uint16_t* b,
                                   const float* h, const int32_t* index, const float* scaling, const uint16_t* dx0,
                                   int M, int N, int K, int R, int L, uint16_t* dx, float* da, float* db,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  begin_call();
  if (int rc = check_lora_shape(M, N, K, R, L)) return rc;
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
  if (int rc = check_lora_shape(M, N, K, R, L)) return rc;
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
  const dim3 grid(static_cast<unsigned>((chunks + 255) / 256)), block(256);
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
