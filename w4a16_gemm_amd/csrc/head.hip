// Entry points of the softmax cross entropy over a quantised vocabulary head
// (w4a16_head.h): argument checks, piece sizes and launches.  Every launch is asynchronous
// on the caller's stream; the only scratch memory is the caller's workspace.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "entry.hpp"
#include "kernels/head.hpp"
#include "w4a16_head.h"

namespace w4a16 {
namespace {

constexpr int kChunkRows = 32768;                       // rows taken at once at most: bounds the workspace
constexpr int64_t kCoeffElements = int64_t{1} << 27;    // coefficients of one piece: 256 MB

int check_head(int M, int N, int K, int group_size, int vocab, int bits) {
  if (M <= 0) return fail(W4A16_ERR_INVALID_ARG, "M must be positive (M=%d)", M);
  if (int rc = check_layer(N, K, group_size, bits)) return rc;
  if (vocab < 1 || vocab > N) return fail(W4A16_ERR_INVALID_ARG, "vocab=%d, not 1..N=%d", vocab, N);
  if (M > kMaxSlots || static_cast<int64_t>(M) * K >= kMaxElements)
    return fail(W4A16_ERR_UNSUPPORTED, "M=%d K=%d: more than 2^27 rows, or 2^31 elements", M, K);
  return W4A16_OK;
}

// Tiles of M rows against `tiles` column tiles of 256.
TileShape pick_rows(int M, int64_t tiles) { return pick_forward(M, 1, static_cast<int>(256 * tiles), false); }

// Rows taken at once: those whose tiles, 64 rows each at least, against all of N one launch takes
// (fewer than kChunkRows from about N = 2^21 on).
int chunk_rows(int M, int N) {
  const int64_t tiles = kMaxBlocks / ceil_div(N, 256);   // 64 or more
  return static_cast<int>(std::min<int64_t>({M, kChunkRows, 64 * (tiles - 1)}));
}

// --- forward ----------------------------------------------------------------------------

struct LossMemory {
  SlotPlan plan;
  MaxSum* part;
  float* label;
  half_t* gathered;
};

LossMemory loss_memory(Carver& ws, int rows, int N, int K, bool act) {
  const int64_t tiles = ceil_div(N, 256);
  LossMemory m;
  m.plan = take_plan(ws, rows, 1, most_tiles(rows, 1, pick_rows(rows, tiles).height), false);
  m.part = ws.take<MaxSum>(static_cast<size_t>(tiles) * rows);
  m.label = ws.take<float>(rows);
  m.gathered = act ? ws.take<half_t>(static_cast<size_t>(rows) * K) : nullptr;
  return m;
}

// Without a plan: the 64-row tiles, for at most 64 rows.
template <int BITS, bool GRAD>
int launch_head(int bm, int64_t row_tiles, hipStream_t st, const half_t* x, int x_rows, bool gathered,
                const Layers& l, const SlotPlan& plan, const HeadRows& rows, const HeadOut& to) {
  auto kern = bm == 64    ? head_low_kernel<BITS, GRAD>
              : bm == 128 ? head_kernel<BITS, GRAD, 128>
                          : head_kernel<BITS, GRAD, 256>;
  const size_t lds = bm == 64 ? low_lds<BITS>() : bm == 128 ? tile_lds<BITS, 128>() : tile_lds<BITS, 256>();
  static const hipError_t ok[3] = {allow_lds(reinterpret_cast<const void*>(head_low_kernel<BITS, GRAD>), low_lds<BITS>()),
                                   allow_lds(reinterpret_cast<const void*>(head_kernel<BITS, GRAD, 128>), tile_lds<BITS, 128>()),
                                   allow_lds(reinterpret_cast<const void*>(head_kernel<BITS, GRAD, 256>), tile_lds<BITS, 256>())};
  if (int rc = lds_status(ok[bm / 128])) return rc;
  const dim3 grid(static_cast<unsigned>(up8(row_tiles * ceil_div(to.v1 - to.v0, 256))));
  hipLaunchKernelGGL(kern, grid, dim3(512), lds, st, x, x_rows, gathered ? 1 : 0, l, plan, rows, to);
  return check_launch("head launch");
}

template <int BITS>
int head_loss(const uint16_t* x, const int32_t* qweight, const uint16_t* scales, const int32_t* qzeros,
              const int32_t* g_idx, int group_size, const int32_t* target, int M, int N, int K, int vocab, float* loss,
              float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  begin_call();
  if (int rc = check_head(M, N, K, group_size, vocab, BITS)) return rc;
  const Buffer bufs[] = {{x, 16, true, "x"},           {qweight, 16, true, "qweight"}, {scales, 16, true, "scales"},
                         {qzeros, 16, false, "qzeros"}, {target, 4, true, "target"},   {loss, 4, true, "loss"},
                         {lse, 4, true, "lse"},         {workspace, 16, true, "workspace"}};
  if (int rc = check_buffers(bufs)) return rc;
  const bool act = g_idx != nullptr;
  const int most = chunk_rows(M, N);
  Carver ws{static_cast<unsigned char*>(workspace)};
  const LossMemory mem = loss_memory(ws, most, N, K, act);
  if (workspace_bytes < ws.used)
    return fail(W4A16_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace_bytes, ws.used);
  hipStream_t st = static_cast<hipStream_t>(stream);
  const Layers l = make_layers(qweight, scales, qzeros, group_size, N, K, BITS, act);
  const TileShape shape = pick_rows(most, ceil_div(N, 256));
  for (int64_t m0 = 0; m0 < M; m0 += most) {
    const int rows = static_cast<int>(std::min<int64_t>(most, M - m0));
    const half_t* hx = reinterpret_cast<const half_t*>(x) + m0 * K;
    // up to 64 rows are ordered by every workgroup itself (37 rows: a launch less, 64 -> 58 us)
    const bool planned = act || M > 64 || shape.bm != 64;
    SlotPlan plan = mem.plan;
    if (planned) run_plan(plan, target + m0, rows, 1, vocab, shape.height, st);
    else plan.counts = nullptr;
    if (act) run_gather(plan, hx, nullptr, l, rows, 1, mem.gathered, st);
    const HeadRows hr{target + m0, mem.label, nullptr};
    const HeadOut to{mem.part, nullptr, 0, 0, vocab, vocab, static_cast<size_t>(rows)};
    const int64_t row_tiles = planned ? most_tiles(rows, 1, shape.height) : 1;
    if (int rc = launch_head<BITS, false>(shape.bm, row_tiles, st, act ? mem.gathered : hx, rows, act, l, plan, hr, to)) return rc;
    hipLaunchKernelGGL(head_join_kernel, dim3(static_cast<unsigned>(ceil_div(rows, 16))), dim3(1024), 0, st, mem.part,
                       static_cast<int>(ceil_div(vocab, 256)), static_cast<size_t>(rows), plan, target + m0, vocab,
                       mem.label, rows, loss + m0, lse + m0);
  }
  return check_launch("head loss launch");
}

// --- backward ---------------------------------------------------------------------------

// A piece of the vocabulary: whole tiles of 256 columns, as many as kCoeffElements hold; the
// tile heights of its logits and of the product of its coefficients with its weights, and the
// most parts of a tile of that product.
struct PieceShape {
  int cols;
  TileShape logits;
  TransposedShape product;
};

PieceShape pick_piece(int rows, int N, int K) {
  PieceShape p;
  const int64_t fit = std::max<int64_t>(1, kCoeffElements / rows / 256) * 256;
  const int64_t pieces = ceil_div(N, fit);
  p.cols = static_cast<int>(ceil_div(ceil_div(N, pieces), 256) * 256);
  p.logits = pick_rows(rows, p.cols / 256);
  p.product = pick_transposed(rows, 1, p.cols, K);
  return p;
}

struct GradMemory {
  SlotPlan plan, logit_plan;
  half_t* coeff;
  float* part;
  float* remainder;
  half_t* gathered;
  int32_t* inverse;
};

GradMemory grad_memory(Carver& ws, int rows, int N, int K, bool act) {
  const PieceShape p = pick_piece(rows, N, K);
  GradMemory m;
  const int height = p.product.height;
  m.plan = take_plan(ws, rows, 1, most_tiles(rows, 1, height), true);
  m.logit_plan = p.logits.height == height ? m.plan : take_plan(ws, rows, 1, most_tiles(rows, 1, p.logits.height), false);
  m.coeff = ws.take<half_t>(static_cast<size_t>(rows) * p.cols);
  m.part = ws.take<float>(static_cast<size_t>(p.product.most) * rows * K);
  m.remainder = ws.take<float>(rows);
  m.gathered = act ? ws.take<half_t>(static_cast<size_t>(rows) * K) : nullptr;
  m.inverse = act ? ws.take<int32_t>(K) : nullptr;
  return m;
}

template <int BITS>
int head_loss_backward(const float* dloss, const uint16_t* x, const int32_t* qweight, const uint16_t* scales,
                       const int32_t* qzeros, const int32_t* g_idx, int group_size, const int32_t* target,
                       const float* lse, int M, int N, int K, int vocab, uint16_t* dx, void* workspace,
                       size_t workspace_bytes, void* stream) {
  begin_call();
  if (int rc = check_head(M, N, K, group_size, vocab, BITS)) return rc;
  const Buffer bufs[] = {{dloss, 4, true, "dloss"},    {x, 16, true, "x"},
                         {qweight, 16, true, "qweight"}, {scales, 16, true, "scales"},
                         {qzeros, 16, false, "qzeros"}, {target, 4, true, "target"},
                         {lse, 4, true, "lse"},         {dx, 16, true, "dx"},
                         {workspace, 16, true, "workspace"}};
  if (int rc = check_buffers(bufs)) return rc;
  const bool act = g_idx != nullptr;
  const int most = chunk_rows(M, N);
  Carver ws{static_cast<unsigned char*>(workspace)};
  const GradMemory mem = grad_memory(ws, most, N, K, act);
  if (workspace_bytes < ws.used)
    return fail(W4A16_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace_bytes, ws.used);
  hipStream_t st = static_cast<hipStream_t>(stream);
  const Layers l = make_layers(qweight, scales, qzeros, group_size, N, K, BITS, act);
  const PieceShape p = pick_piece(most, N, K);
  if (act) run_invert(l, 1, mem.inverse, st);
  for (int64_t m0 = 0; m0 < M; m0 += most) {
    const int rows = static_cast<int>(std::min<int64_t>(most, M - m0));
    const half_t* hx = reinterpret_cast<const half_t*>(x) + m0 * K;
    const int height = p.product.height;
    run_plan(mem.plan, target + m0, rows, 1, vocab, height, st);
    if (p.logits.height != height) run_plan(mem.logit_plan, target + m0, rows, 1, vocab, p.logits.height, st);
    if (act) run_gather(mem.plan, hx, nullptr, l, rows, 1, mem.gathered, st);
    const HeadRows hr{target + m0, mem.remainder, lse + m0};
    for (int v0 = 0; v0 < vocab; v0 += p.cols) {
      // padding columns up to a whole load of zero points have the coefficient 0
      const int v1 = static_cast<int>(std::min<int64_t>(int64_t{v0} + p.cols, std::min<int64_t>(ceil_div(vocab, 16) * 16, N)));
      const HeadOut to{nullptr, mem.coeff, p.cols, v0, v1, vocab, static_cast<size_t>(rows)};
      if (int rc = launch_head<BITS, true>(p.logits.bm, most_tiles(rows, 1, p.logits.height), st, act ? mem.gathered : hx, rows, act, l,
                                           mem.logit_plan, hr, to))
        return rc;
      const TOut out{nullptr, nullptr, mem.part, static_cast<size_t>(rows), v0 > 0};
      if (int rc = run_transposed(BITS, p.product.bm, most_tiles(rows, 1, height), mem.coeff, rows, p.cols, true, l, mem.plan, rows, v0, v1, vocab,
                                  p.cols, p.product.most, out, st))
        return rc;
    }
    hipLaunchKernelGGL(head_dx_kernel<BITS>, dim3(rows), dim3(256), 0, st, mem.part, static_cast<size_t>(rows),
                       p.product.most, tile_slots(p.product.bm), p.cols, mem.plan, l, act ? mem.inverse : nullptr, target + m0, mem.remainder, dloss + m0,
                       reinterpret_cast<half_t*>(dx) + m0 * K);
  }
  return check_launch("head backward launch");
}

}  // namespace
}  // namespace w4a16

using namespace w4a16;

extern "C" {

size_t w4a16_head_loss_workspace(int M, int N, int K, int act_order) {
  const bool ok = check_head(M, N, K, K, N, 4) == W4A16_OK;
  clear_error();
  if (!ok) return 0;
  Carver ws{nullptr};
  loss_memory(ws, chunk_rows(M, N), N, K, act_order != 0);
  return ws.used;
}

int w4a16_head_loss(const uint16_t* x, const int32_t* qweight, const uint16_t* scales, const int32_t* qzeros,
                    const int32_t* g_idx, int group_size, const int32_t* target, int M, int N, int K, int vocab,
                    float* loss, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  return head_loss<4>(x, qweight, scales, qzeros, g_idx, group_size, target, M, N, K, vocab, loss, lse, workspace,
                      workspace_bytes, stream);
}

int w8a16_head_loss(const uint16_t* x, const int32_t* qweight, const uint16_t* scales, const int32_t* qzeros,
                    const int32_t* g_idx, int group_size, const int32_t* target, int M, int N, int K, int vocab,
                    float* loss, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  return head_loss<8>(x, qweight, scales, qzeros, g_idx, group_size, target, M, N, K, vocab, loss, lse, workspace,
                      workspace_bytes, stream);
}

size_t w4a16_head_loss_backward_workspace(int M, int N, int K, int act_order) {
  const bool ok = check_head(M, N, K, K, N, 4) == W4A16_OK;
  clear_error();
  if (!ok) return 0;
  Carver ws{nullptr};
  grad_memory(ws, chunk_rows(M, N), N, K, act_order != 0);
  return ws.used;
}

int w4a16_head_loss_backward(const float* dloss, const uint16_t* x, const int32_t* qweight, const uint16_t* scales,
                             const int32_t* qzeros, const int32_t* g_idx, int group_size, const int32_t* target,
                             const float* lse, int M, int N, int K, int vocab, uint16_t* dx, void* workspace,
                             size_t workspace_bytes, void* stream) {
  return head_loss_backward<4>(dloss, x, qweight, scales, qzeros, g_idx, group_size, target, lse, M, N, K, vocab, dx,
                               workspace, workspace_bytes, stream);
}

int w8a16_head_loss_backward(const float* dloss, const uint16_t* x, const int32_t* qweight, const uint16_t* scales,
                             const int32_t* qzeros, const int32_t* g_idx, int group_size, const int32_t* target,
                             const float* lse, int M, int N, int K, int vocab, uint16_t* dx, void* workspace,
                             size_t workspace_bytes, void* stream) {
  return head_loss_backward<8>(dloss, x, qweight, scales, qzeros, g_idx, group_size, target, lse, M, N, K, vocab, dx,
                               workspace, workspace_bytes, stream);
}

}  // extern "C"
