// Entry points of the mixtures of experts (w4a16_experts.h): argument checks, kernel choice
// and launches.  Every launch is asynchronous on the caller's stream; the only scratch
// memory is the caller's workspace.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "entry.hpp"
#include "kernels/experts.hpp"
#include "kernels/few.hpp"
#include "kernels/low.hpp"
#include "kernels/route.hpp"
#include "kernels/slots.hpp"
#include "kernels/transposed.hpp"
#include "w4a16_experts.h"

namespace w4a16 {

void run_plan(const SlotPlan& p, const int32_t* index, int S, int E, int limit, int height, hipStream_t st) {
  const size_t row = sizeof(int32_t) * (E + 1);
  const int blocks = plan_blocks(S);
  if (blocks == 1) {
    hipLaunchKernelGGL(plan_slots_kernel, dim3(1), dim3(kPlanThreads), kPlanWaves * row, st, index, S, E, limit, height, p);
    return;
  }
  const int per = static_cast<int>((static_cast<int64_t>(S) + blocks - 1) / blocks);
  hipLaunchKernelGGL(plan_count_kernel, dim3(blocks), dim3(kPlanThreads), row, st, index, S, per, E, limit, p.sums);
  hipLaunchKernelGGL(plan_scan_kernel, dim3(1), dim3(kPlanThreads), 0, st, blocks, E, height, p, p.sums);
  hipLaunchKernelGGL(plan_place_kernel, dim3(blocks), dim3(kPlanThreads), kPlanWaves * row, st, index, S, per, E, limit,
                     height, blocks, p, p.sums);
}

void run_gather(const SlotPlan& p, const half_t* x, const int32_t* index, const Layers& l, int S, int T, half_t* out,
                hipStream_t st) {
  hipLaunchKernelGGL(gather_slots_kernel, dim3(S), dim3(256), 0, st, x, index, p, l, T, out);
}

void run_invert(const Layers& l, int E, int32_t* inverse, hipStream_t st) {
  hipLaunchKernelGGL(invert_order_kernel, dim3(static_cast<unsigned>(ceil_div(l.K, 256)), E), dim3(256), 0, st, l, inverse);
}

namespace {

template <int BITS, int BM>
int launch_transposed(int64_t tiles, const half_t* a, int a_rows, int a_pitch, bool by_place, const Layers& l,
                      const SlotPlan& p, int slots, int n_begin, int n_end, int n_valid, int n_most, int most,
                      const TOut& to, hipStream_t st) {
  auto kern = transposed_kernel<BITS, BM>;
  constexpr size_t lds = transposed_lds<BITS, BM>();
  static const hipError_t lds_ok = allow_lds(reinterpret_cast<const void*>(kern), lds);
  if (int rc = lds_status(lds_ok)) return rc;
  const dim3 grid(static_cast<unsigned>(piece_blocks(tiles * ceil_div(l.K, 256), tile_slots(BM))));
  hipLaunchKernelGGL(kern, grid, dim3(512), lds, st, a, a_rows, a_pitch, by_place ? 1 : 0, l, p, slots, n_begin, n_end,
                     n_valid, n_most, most, to);
  return check_launch("transposed launch");
}

}  // namespace

int run_transposed(int bits, int bm, int64_t tiles, const half_t* a, int a_rows, int a_pitch, bool by_place,
                   const Layers& l, const SlotPlan& p, int slots, int n_begin, int n_end, int n_valid, int n_most, int most,
                   const TOut& to, hipStream_t st) {
  auto launch = bits == 4 ? (bm == 256 ? launch_transposed<4, 256> : launch_transposed<4, 128>)
                          : (bm == 256 ? launch_transposed<8, 256> : launch_transposed<8, 128>);
  return launch(tiles, a, a_rows, a_pitch, by_place, l, p, slots, n_begin, n_end, n_valid, n_most, most, to, st);
}

namespace {

int check_experts(int M, int T, int E, int N, int K, int group_size, int bits) {
  if (M <= 0 || T <= 0) return fail(W4A16_ERR_INVALID_ARG, "M and T must be positive (M=%d T=%d)", M, T);
  if (E < 1 || E > kMaxExperts) return fail(W4A16_ERR_UNSUPPORTED, "%d experts, not 1..%d", E, kMaxExperts);
  if (static_cast<int64_t>(M) * T > kMaxSlots)
    return fail(W4A16_ERR_UNSUPPORTED, "M=%d T=%d: more than 2^27 slots", M, T);
  return check_layer(N, K, group_size, bits);
}

// --- tile shapes ----------------------------------------------------------------------

// Tiles of 64 columns against 256, K 4096: 300 rows of one expert, N 4096 40.0 / 43.0 us, 128 of
// two 8-bit experts, N 1024 37.2 / 51.4 us.
TileShape pick_shape(int64_t S, int E, int cols) { return pick_forward(S, E, cols, true); }

// --- forward ----------------------------------------------------------------------------

// Few rows per expert: the streaming kernel, at most 4096 channels per walk over its
// wavefronts (16 of them with up to 2 steps of 128 channels, without a spill; 3 and 4 steps spill 11
// to 48 registers, and the 2 steps of a longer row 5 to 15, outside the loop over the units).
// Up to 16 rows on average, and up to 32, which are two of its tiles and read the codes twice,
// where the 64-row tiles would leave half of the compute units idle.  Against those tiles (K
// 4096): 16 experts, N 4096, of 16 / 24 rows 34 / 54 us, in tiles 43 / 44 us; 8 of 16 / 24 / 32 rows 22 /
// 31 / 33 us, in tiles 39 / 40 / 40 us; 8, N 14336, 53 / 84 / 91 us, in tiles 63 / 64 / 64 us.
struct FewShape {
  bool ok;
  int waves, steps, chunks;
};

FewShape pick_few(int64_t S, int E, int N, int K) {
  FewShape f{};
  const int64_t used = std::min<int64_t>(E, S);
  f.ok = S <= kFewSlots && (S <= 16 * used || (S <= 32 * used && used * ceil_div(N, 256) <= kUnits / 2));
  const int total = static_cast<int>(ceil_div(K, 128));
  f.chunks = static_cast<int>(ceil_div(total, 32));
  const int walk = static_cast<int>(ceil_div(total, f.chunks));
  f.steps = static_cast<int>(ceil_div(walk, 16));
  f.waves = static_cast<int>(ceil_div(walk, f.steps));
  return f;
}

struct ForwardMemory {
  SlotPlan plan;
  half_t* gathered;
};

ForwardMemory forward_memory(Carver& ws, int64_t S, int E, int N, int K, bool act, int height) {
  ForwardMemory m{};
  if (!pick_few(S, E, N, K).ok) m.plan = take_plan(ws, S, E, most_tiles(S, E, height), false);
  m.gathered = act ? ws.take<half_t>(static_cast<size_t>(S) * K) : nullptr;
  return m;
}

int check_forward(int M, int T, int E, int N, int K, bool act) {
  const int64_t S = static_cast<int64_t>(M) * T;
  if ((act ? S : M) * static_cast<int64_t>(K) >= kMaxElements)
    return fail(W4A16_ERR_UNSUPPORTED, "M=%d T=%d K=%d: 2^31 elements or more", M, T, K);
  const TileShape shape = pick_shape(S, E, N);
  if (most_tiles(S, E, shape.height) * ceil_div(N, 64 * shape.nb) > kMaxBlocks || (act && S > 2 * kMaxBlocks))
    return fail(W4A16_ERR_UNSUPPORTED, "M=%d T=%d N=%d: more tiles than one launch takes", M, T, N);
  return W4A16_OK;
}

template <int NB, int BITS, int BM>
int launch_forward(dim3 grid, hipStream_t st, const half_t* x, int x_rows, int gathered, int S, int T, const Layers& l,
                   const SlotPlan& plan, half_t* y) {
  auto kern = experts_gemm_kernel<NB, BITS, BM>;
  constexpr size_t lds = tile_lds<BITS, BM>();
  static const hipError_t lds_ok = allow_lds(reinterpret_cast<const void*>(kern), lds);
  if (int rc = lds_status(lds_ok)) return rc;
  hipLaunchKernelGGL(kern, grid, dim3(512), lds, st, x, x_rows, gathered, S, T, l, plan, y);
  return check_launch("experts launch");
}

template <int STEPS, int BITS, bool LONG, bool WAVE>
int launch_few_t(const FewShape& f, hipStream_t st, const half_t* x, int by_slot, int T, const int32_t* index, int S,
                 int E, const Layers& l, half_t* y) {
  auto kern = experts_few_kernel<STEPS, BITS, LONG, WAVE>;
  static const hipError_t lds_ok = allow_lds(reinterpret_cast<const void*>(kern), few_lds<WAVE>(16));
  if (int rc = lds_status(lds_ok)) return rc;
  hipLaunchKernelGGL(kern, dim3(kUnits), dim3(64 * f.waves), few_lds<WAVE>(f.waves), st, x, by_slot, T, index, S, E, l,
                     f.chunks, y);
  return check_launch("experts launch");
}

template <int BITS, bool WAVE>
int launch_few(const FewShape& f, hipStream_t st, const half_t* x, int by_slot, int T, const int32_t* index, int S, int E,
               const Layers& l, half_t* y) {
  if (f.chunks > 1) return launch_few_t<2, BITS, true, WAVE>(f, st, x, by_slot, T, index, S, E, l, y);   // 17 or more steps
  if (f.steps == 1) return launch_few_t<1, BITS, false, WAVE>(f, st, x, by_slot, T, index, S, E, l, y);
  return launch_few_t<2, BITS, false, WAVE>(f, st, x, by_slot, T, index, S, E, l, y);
}

template <int BITS>
int experts_gemm(const uint16_t* x, const int32_t* qweight, const uint16_t* scales, const int32_t* qzeros,
                 const int32_t* g_idx, int group_size, const int32_t* index, int M, int T, int E, int N, int K,
                 uint16_t* y, void* workspace, size_t workspace_bytes, void* stream) {
  begin_call();
  if (int rc = check_experts(M, T, E, N, K, group_size, BITS)) return rc;
  const Buffer bufs[] = {{x, 16, true, "x"},          {qweight, 16, true, "qweight"}, {scales, 16, true, "scales"},
                         {qzeros, 16, false, "qzeros"}, {index, 4, true, "index"},    {y, 16, true, "y"},
                         {workspace, 16, false, "workspace"}};
  if (int rc = check_buffers(bufs)) return rc;
  const bool act = g_idx != nullptr;
  if (int rc = check_forward(M, T, E, N, K, act)) return rc;
  const int S = M * T;
  const TileShape shape = pick_shape(S, E, N);
  Carver ws{static_cast<unsigned char*>(workspace)};
  const ForwardMemory mem = forward_memory(ws, S, E, N, K, act, shape.height);
  if (!workspace && ws.used > 0) return fail(W4A16_ERR_INVALID_ARG, "NULL buffer workspace");
  if (workspace_bytes < ws.used)
    return fail(W4A16_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace_bytes, ws.used);
  hipStream_t st = static_cast<hipStream_t>(stream);
  const Layers l = make_layers(qweight, scales, qzeros, group_size, N, K, BITS, act);
  const half_t* hx = reinterpret_cast<const half_t*>(x);
  const FewShape few = pick_few(S, E, N, K);
  if (few.ok) {
    if (act) hipLaunchKernelGGL(gather_rows_kernel, dim3(S), dim3(256), 0, st, hx, index, E, l, T, mem.gathered);
    auto launch = S <= 64 ? launch_few<BITS, true> : launch_few<BITS, false>;
    return launch(few, st, act ? mem.gathered : hx, act, T, index, S, E, l, reinterpret_cast<half_t*>(y));
  }
  run_plan(mem.plan, index, S, E, E, shape.height, st);
  if (act)
    run_gather(mem.plan, hx, index, l, S, T, mem.gathered, st);
  const dim3 grid(static_cast<unsigned>(up8(most_tiles(S, E, shape.height) * ceil_div(N, 64 * shape.nb))));
  const half_t* rows = act ? mem.gathered : hx;
  half_t* hy = reinterpret_cast<half_t*>(y);
  if (shape.bm == 64) {
    static const hipError_t lds_ok = allow_lds(reinterpret_cast<const void*>(experts_low_kernel<BITS>), low_lds<BITS>());
    if (int rc = lds_status(lds_ok)) return rc;
    hipLaunchKernelGGL(experts_low_kernel<BITS>, grid, dim3(512), low_lds<BITS>(), st, rows, act ? S : M, act ? 1 : 0, S, T, l,
                       mem.plan, hy);
    return check_launch("experts launch");
  }
  auto launch = shape.nb == 4 ? (shape.bm == 256 ? launch_forward<4, BITS, 256> : launch_forward<4, BITS, 128>)
                              : launch_forward<1, BITS, 256>;
  return launch(grid, st, rows, act ? S : M, act, S, T, l, mem.plan, hy);
}

// --- backward ---------------------------------------------------------------------------

struct BackwardMemory {
  SlotPlan plan;
  float* part;        // NULL: straight to dx
  int32_t* inverse;   // act order
};

// Sums go to dx themselves where a row has one slot and its channels their own order;
// partial sums are kept for the tiles that are in parts.
bool is_direct(int T, bool act) { return T == 1 && !act; }

BackwardMemory backward_memory(Carver& ws, int64_t S, int T, int E, int K, bool act, const TransposedShape& shape) {
  BackwardMemory m;
  const bool parts = !is_direct(T, act) || shape.most > 1;
  m.plan = take_plan(ws, S, E, most_tiles(S, E, shape.height), parts);
  m.part = parts ? ws.take<float>(static_cast<size_t>(shape.most) * S * K) : nullptr;
  m.inverse = act ? ws.take<int32_t>(static_cast<size_t>(E) * K) : nullptr;
  return m;
}

int check_backward(int M, int T, int E, int N, int K, bool act) {
  const int64_t S = static_cast<int64_t>(M) * T;
  if (S * N >= kMaxElements) return fail(W4A16_ERR_UNSUPPORTED, "M=%d T=%d N=%d: 2^31 elements or more", M, T, N);
  const TransposedShape shape = pick_transposed(S, E, N, K);
  if (piece_blocks(most_tiles(S, E, shape.height) * ceil_div(K, 256), 64) > kMaxBlocks || (!is_direct(T, act) && M > kMaxBlocks))
    return fail(W4A16_ERR_UNSUPPORTED, "M=%d T=%d K=%d: more tiles or sums than one launch takes", M, T, K);
  return W4A16_OK;
}

template <int BITS>
int launch_backward(const uint16_t* dy, const int32_t* qweight, const uint16_t* scales, const int32_t* qzeros, bool act,
                    int group_size, const int32_t* index, const uint16_t* dx0, int M, int T, int E, int N, int K,
                    uint16_t* dx, void* workspace, size_t workspace_bytes, void* stream) {
  if (int rc = check_backward(M, T, E, N, K, act)) return rc;
  const int S = M * T;
  const TransposedShape shape = pick_transposed(S, E, N, K);
  Carver ws{static_cast<unsigned char*>(workspace)};
  const BackwardMemory mem = backward_memory(ws, S, T, E, K, act, shape);
  if (workspace_bytes < ws.used)
    return fail(W4A16_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace_bytes, ws.used);
  hipStream_t st = static_cast<hipStream_t>(stream);
  const Layers l = make_layers(qweight, scales, qzeros, group_size, N, K, BITS, act);
  const bool direct = is_direct(T, act);
  run_plan(mem.plan, index, S, E, E, shape.height, st);
  const half_t* h0 = reinterpret_cast<const half_t*>(dx0);
  half_t* hx = reinterpret_cast<half_t*>(dx);
  const TOut to{direct ? hx : nullptr, direct ? h0 : nullptr, mem.part, static_cast<size_t>(S), 0};
  if (int rc = run_transposed(BITS, shape.bm, most_tiles(S, E, shape.height), reinterpret_cast<const half_t*>(dy), S, N, false, l,
                              mem.plan, S, 0, N, N, N, shape.most, to, st))
    return rc;
  if (mem.part) {
    if (act) {
      run_invert(l, E, mem.inverse, st);
      hipLaunchKernelGGL(sum_ordered_kernel, dim3(M), dim3(512), 0, st, mem.part, static_cast<size_t>(S), shape.most, tile_slots(shape.bm), N, T,
                         index, E, mem.plan, mem.inverse, K, h0, hx);
    } else {
      hipLaunchKernelGGL(sum_slots_kernel, dim3(M), dim3(256), 0, st, mem.part, static_cast<size_t>(S), shape.most, tile_slots(shape.bm), N, T,
                         index, E, mem.plan, K, direct ? 1 : 0, h0, hx);
    }
  }
  return check_launch("experts backward launch");
}

template <int BITS>
int experts_backward(const uint16_t* dy, const int32_t* qweight, const uint16_t* scales, const int32_t* qzeros,
                     const int32_t* g_idx, int group_size, const int32_t* index, bool with_index, const uint16_t* dx0,
                     int M, int T, int E, int N, int K, uint16_t* dx, void* workspace, size_t workspace_bytes,
                     void* stream) {
  begin_call();
  if (int rc = check_experts(M, T, E, N, K, group_size, BITS)) return rc;
  const Buffer bufs[] = {{dy, 16, true, "dy"},          {qweight, 16, true, "qweight"},
                         {scales, 16, true, "scales"},  {qzeros, 16, false, "qzeros"},
                         {index, 4, with_index, "index"}, {dx0, 16, false, "dx0"},
                         {dx, 16, true, "dx"},          {workspace, 16, true, "workspace"}};
  if (int rc = check_buffers(bufs)) return rc;
  return launch_backward<BITS>(dy, qweight, scales, qzeros, g_idx != nullptr, group_size, index, dx0, M, T, E, N, K, dx,
                               workspace, workspace_bytes, stream);
}

// --- routing ----------------------------------------------------------------------------

int check_route(int logit_bits, int M, int E, int top_k) {
  if (M <= 0 || top_k <= 0) return fail(W4A16_ERR_INVALID_ARG, "M and top_k must be positive (M=%d top_k=%d)", M, top_k);
  if (logit_bits != 16 && logit_bits != 32) return fail(W4A16_ERR_UNSUPPORTED, "logits of %d bits, not 16 or 32", logit_bits);
  if (E < 1 || E > kMaxExperts) return fail(W4A16_ERR_UNSUPPORTED, "%d experts, not 1..%d", E, kMaxExperts);
  if (top_k > E) return fail(W4A16_ERR_INVALID_ARG, "top_k=%d of %d experts", top_k, E);
  // 2^23 workgroups of 256 threads
  if (M > (E <= 128 ? kMaxSlots : kMaxSlots / 4)) return fail(W4A16_ERR_UNSUPPORTED, "M=%d E=%d: too many rows for one launch", M, E);
  return W4A16_OK;
}

// Sixteen lanes per row up to 128 experts, a wavefront above.
template <typename F>
void by_experts(int M, int E, F launch) {
  const auto blocks = [&](int lanes) { return dim3(static_cast<unsigned>(ceil_div(M, 256 / lanes))); };
  if (E <= 16) launch(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{}, blocks(16));
  else if (E <= 64) launch(std::integral_constant<int, 16>{}, std::integral_constant<int, 4>{}, blocks(16));
  else if (E <= 128) launch(std::integral_constant<int, 16>{}, std::integral_constant<int, 8>{}, blocks(16));
  else if (E <= 256) launch(std::integral_constant<int, 64>{}, std::integral_constant<int, 4>{}, blocks(64));
  else launch(std::integral_constant<int, 64>{}, std::integral_constant<int, 8>{}, blocks(64));
}

int check_combine(int M, int T, int N) {
  if (M <= 0 || T <= 0 || N <= 0) return fail(W4A16_ERR_INVALID_ARG, "sizes must be positive: M=%d T=%d N=%d", M, T, N);
  if (N % 8 != 0) return fail(W4A16_ERR_INVALID_ARG, "N=%d is not a multiple of 8", N);
  if (static_cast<int64_t>(M) * N >= int64_t{1} << 34 || static_cast<int64_t>(M) * T > kMaxSlots || N > kMaxOutputs)
    return fail(W4A16_ERR_UNSUPPORTED, "M=%d T=%d N=%d: too large for one launch", M, T, N);
  return W4A16_OK;
}

}  // namespace
}  // namespace w4a16

using namespace w4a16;

extern "C" {

int w4a16_route(const void* logits, int logit_bits, int M, int E, int top_k, int renormalise, int32_t* index,
                float* weights, void* stream) {
  begin_call();
  if (int rc = check_route(logit_bits, M, E, top_k)) return rc;
  const Buffer bufs[] = {{logits, 4, true, "logits"}, {index, 4, true, "index"}, {weights, 4, true, "weights"}};
  if (int rc = check_buffers(bufs)) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  by_experts(M, E, [&](auto lanes, auto per, dim3 grid) {
    if (logit_bits == 16)
      hipLaunchKernelGGL((route_kernel<lanes.value, per.value, half_t>), grid, dim3(256), 0, st,
                         static_cast<const half_t*>(logits), M, E, top_k, renormalise != 0, index, weights);
    else
      hipLaunchKernelGGL((route_kernel<lanes.value, per.value, float>), grid, dim3(256), 0, st,
                         static_cast<const float*>(logits), M, E, top_k, renormalise != 0, index, weights);
  });
  return check_launch("route launch");
}

int w4a16_route_backward(const float* dweights, const void* logits, int logit_bits, const int32_t* index,
                         const float* weights, int M, int E, int top_k, int renormalise, void* dlogits, void* stream) {
  begin_call();
  if (int rc = check_route(logit_bits, M, E, top_k)) return rc;
  const Buffer bufs[] = {{dweights, 4, true, "dweights"}, {logits, 4, true, "logits"},   {index, 4, true, "index"},
                         {weights, 4, true, "weights"},   {dlogits, 4, true, "dlogits"}};
  if (int rc = check_buffers(bufs)) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  by_experts(M, E, [&](auto lanes, auto per, dim3 grid) {
    if (logit_bits == 16)
      hipLaunchKernelGGL((route_backward_kernel<lanes.value, per.value, half_t>), grid, dim3(256), 0, st, dweights,
                         static_cast<const half_t*>(logits), index, weights, M, E, top_k, renormalise != 0,
                         static_cast<half_t*>(dlogits));
    else
      hipLaunchKernelGGL((route_backward_kernel<lanes.value, per.value, float>), grid, dim3(256), 0, st, dweights,
                         static_cast<const float*>(logits), index, weights, M, E, top_k, renormalise != 0,
                         static_cast<float*>(dlogits));
  });
  return check_launch("route backward launch");
}

size_t w4a16_experts_gemm_workspace(int M, int T, int E, int N, int K, int act_order) {
  const bool ok = check_experts(M, T, E, N, K, K, 4) == W4A16_OK && check_forward(M, T, E, N, K, act_order != 0) == W4A16_OK;
  clear_error();
  if (!ok) return 0;
  Carver ws{nullptr};
  const int64_t S = static_cast<int64_t>(M) * T;
  forward_memory(ws, S, E, N, K, act_order != 0, pick_shape(S, E, N).height);
  return ws.used;
}

int w4a16_experts_gemm(const uint16_t* x, const int32_t* qweight, const uint16_t* scales, const int32_t* qzeros,
                       const int32_t* g_idx, int group_size, const int32_t* index, int M, int T, int E, int N, int K,
                       uint16_t* y, void* workspace, size_t workspace_bytes, void* stream) {
  return experts_gemm<4>(x, qweight, scales, qzeros, g_idx, group_size, index, M, T, E, N, K, y, workspace,
                         workspace_bytes, stream);
}

int w8a16_experts_gemm(const uint16_t* x, const int32_t* qweight, const uint16_t* scales, const int32_t* qzeros,
                       const int32_t* g_idx, int group_size, const int32_t* index, int M, int T, int E, int N, int K,
                       uint16_t* y, void* workspace, size_t workspace_bytes, void* stream) {
  return experts_gemm<8>(x, qweight, scales, qzeros, g_idx, group_size, index, M, T, E, N, K, y, workspace,
                         workspace_bytes, stream);
}

size_t w4a16_experts_backward_workspace(int M, int T, int E, int N, int K, int act_order) {
  const bool ok = check_experts(M, T, E, N, K, K, 4) == W4A16_OK && check_backward(M, T, E, N, K, act_order != 0) == W4A16_OK;
  clear_error();
  if (!ok) return 0;
  Carver ws{nullptr};
  const int64_t S = static_cast<int64_t>(M) * T;
  backward_memory(ws, S, T, E, K, act_order != 0, pick_transposed(S, E, N, K));
  return ws.used;
}

int w4a16_experts_backward(const uint16_t* dy, const int32_t* qweight, const uint16_t* scales, const int32_t* qzeros,
                           const int32_t* g_idx, int group_size, const int32_t* index, const uint16_t* dx0, int M, int T,
                           int E, int N, int K, uint16_t* dx, void* workspace, size_t workspace_bytes, void* stream) {
  return experts_backward<4>(dy, qweight, scales, qzeros, g_idx, group_size, index, true, dx0, M, T, E, N, K, dx,
                             workspace, workspace_bytes, stream);
}

int w8a16_experts_backward(const uint16_t* dy, const int32_t* qweight, const uint16_t* scales, const int32_t* qzeros,
                           const int32_t* g_idx, int group_size, const int32_t* index, const uint16_t* dx0, int M, int T,
                           int E, int N, int K, uint16_t* dx, void* workspace, size_t workspace_bytes, void* stream) {
  return experts_backward<8>(dy, qweight, scales, qzeros, g_idx, group_size, index, true, dx0, M, T, E, N, K, dx,
                             workspace, workspace_bytes, stream);
}

int w4a16_gemm_backward(const uint16_t* dy, const int32_t* qweight, const uint16_t* scales, const int32_t* qzeros,
                        const int32_t* g_idx, int group_size, const uint16_t* dx0, int M, int N, int K, uint16_t* dx,
                        void* workspace, size_t workspace_bytes, void* stream) {
  return experts_backward<4>(dy, qweight, scales, qzeros, g_idx, group_size, nullptr, false, dx0, M, 1, 1, N, K, dx,
                             workspace, workspace_bytes, stream);
}

int w8a16_gemm_backward(const uint16_t* dy, const int32_t* qweight, const uint16_t* scales, const int32_t* qzeros,
                        const int32_t* g_idx, int group_size, const uint16_t* dx0, int M, int N, int K, uint16_t* dx,
                        void* workspace, size_t workspace_bytes, void* stream) {
  return experts_backward<8>(dy, qweight, scales, qzeros, g_idx, group_size, nullptr, false, dx0, M, 1, 1, N, K, dx,
                             workspace, workspace_bytes, stream);
}

int w4a16_experts_combine(const uint16_t* y, const float* weights, int M, int T, int N, uint16_t* out, void* stream) {
  begin_call();
  if (int rc = check_combine(M, T, N)) return rc;
  const Buffer bufs[] = {{y, 16, true, "y"}, {weights, 4, true, "weights"}, {out, 16, true, "out"}};
  if (int rc = check_buffers(bufs)) return rc;
  const int64_t runs = static_cast<int64_t>(M) * (N / 8);
  hipLaunchKernelGGL(combine_kernel, dim3(static_cast<unsigned>(ceil_div(runs, 256))), dim3(256), 0,
                     static_cast<hipStream_t>(stream), reinterpret_cast<const half_t*>(y), weights, runs, T, N,
                     reinterpret_cast<half_t*>(out));
  return check_launch("combine launch");
}

int w4a16_experts_combine_backward(const uint16_t* dout, const uint16_t* y, const float* weights, int M, int T, int N,
                                   uint16_t* dy, float* dweights, void* stream) {
  begin_call();
  if (int rc = check_combine(M, T, N)) return rc;
  if (M > 1 << 23) return fail(W4A16_ERR_UNSUPPORTED, "M=%d: at most 2^23 rows", M);
  const Buffer bufs[] = {{dout, 16, true, "dout"}, {y, 16, true, "y"}, {weights, 4, true, "weights"},
                         {dy, 16, true, "dy"},     {dweights, 4, true, "dweights"}};
  if (int rc = check_buffers(bufs)) return rc;
  hipLaunchKernelGGL(combine_backward_kernel, dim3(M), dim3(256), 0, static_cast<hipStream_t>(stream),
                     reinterpret_cast<const half_t*>(dout), reinterpret_cast<const half_t*>(y), weights, T, N,
                     reinterpret_cast<half_t*>(dy), dweights);
  return check_launch("combine backward launch");
}

}  // extern "C"
