/*
 * w4a16_experts.h -- C ABI of mixtures of experts of the quantised layer (gfx950): routing of
 * rows to experts, products with the experts' packed weights, the products back through
 * them, and the weighted sum of the experts' outputs.
 *
 * The experts' weights are frozen in 4 or 8 bits; what is trained are adapters beside them
 * (w4a16_adapters.h) and what comes before them, so the gradients here are those of the
 * activations and of the routing.  Part of libw4a16.so; statuses, w4a16_last_error and the
 * conventions of w4a16.h apply: device pointers, everything asynchronous and ordered on
 * `stream`, the stream belongs to the current device, no exception crosses the ABI, nothing
 * is launched on failure.  No call allocates, so every call can be captured into a graph.
 *
 * Shapes: M rows, T experts per row, S = M T slots, E experts (1 .. 512), N output and K input
 * channels; M, T > 0, S <= 2^27.  The layers' shapes are those of w4a16.h and besides K % 64
 * == 0, for 8-bit weights N % 16 == 0, N <= 2^24, fewer than 2^32 bytes of codes per expert, and
 * fewer than 2^31 elements of x, of dy and of the slots' rows of K channels under act order;
 * what one launch takes bounds S to 2^23 under act order, M to 2^22 where the gradients
 * of several slots are summed or act order is undone, and the tiles of a product
 * (about S / 256 + E row tiles of N / 256 columns, back K / 256) to 2^22.
 *   qweight   int32 [E][w4a16_qweight_words(N, K, act_order)] (w8a16: its own function): the
 *             experts' weight buffers one after the other
 *   scales    binary16 [E][G][N];  qzeros  int32 [E][G][N/8] (8 bits: [N/4]) or NULL: symmetric
 *   g_idx     int32 [E][K] or NULL: act order, every expert its own (only its presence counts)
 *   index     int32 [M][T]: expert of every slot.  A value outside [0, E) (-1 by convention) is
 *             a slot without an expert: padding, or a row that the router left short.
 *   weights   float [M][T]
 *   workspace 16-byte aligned device memory of at least the size that the matching _workspace
 *             function returns for the same sizes (0 on sizes that both widths refuse, or where
 *             none is needed: workspace may then be NULL), owned by
 *             the caller and free again once the stream has passed the call.  Calls that may
 *             run at once, two graphs for instance, need a workspace each.
 * Buffers must be 16-byte aligned (index, weights, dweights, logits, dlogits: 4-byte aligned).
 * Outputs must not overlap inputs or the workspace, but for dx and dx0.
 * W^ = binary16((q - Z) S), the values of w4a16_dequant, in both directions; sums are fp32 in
 * a fixed order: the same call gives the same bits.  A row's results do not depend on the
 * values of other rows.
 */
#ifndef W4A16_EXPERTS_H
#define W4A16_EXPERTS_H

#include "w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Routes every row to its top_k experts: p = softmax(logits[m]) in fp32, index[m] = the
 * experts of the top_k largest logits in descending order, of equal ones the lower index
 * first, weights[m][t] = p of that expert, divided by the sum of the row's weights where
 * renormalise != 0.  An expert whose logit is -infinity (masked) or NaN is never chosen; where
 * fewer than top_k are left, the rest of the row gets index -1 and weight 0.  A NaN or +infinity
 * in a row makes the weights of its chosen experts NaN.
 *   logits [M][E], binary16 (logit_bits 16) or float (32);  1 <= top_k <= E <= 512; M <= 2^27
 *   (2^25 above 128 experts)
 *   index  out int32 [M][top_k];  weights out float [M][top_k]
 * Errors: INVALID_ARG, UNSUPPORTED (E, logit_bits, M), MISALIGNED, HIP. */
int w4a16_route(const void* logits, int logit_bits, int M, int E, int top_k, int renormalise, int32_t* index,
                float* weights, void* stream);

/* Gradient of the logits for that of the weights, dweights float [M][top_k]; logits, index and
 * weights as w4a16_route took and gave them.  dlogits out: logits' type.  Renormalised:
 * dl = w (dw - sum w dw) for the chosen, 0 for the others; else dl_j = [j chosen] w dw - p_j sum
 * w dw.  Slots with an index outside [0, E) take no part.  Errors as w4a16_route. */
int w4a16_route_backward(const float* dweights, const void* logits, int logit_bits, const int32_t* index,
                         const float* weights, int M, int E, int top_k, int renormalise, void* dlogits, void* stream);

/* Workspace bytes of w4a16_experts_gemm and w8a16_experts_gemm.  act_order: 1 where g_idx is
 * not NULL. */
size_t w4a16_experts_gemm_workspace(int M, int T, int E, int N, int K, int act_order);

/* y[m][t] = binary16(W^_e x[m]), e = index[m][t]: binary16 operands, fp32 sums, one rounding.
 * Slots without an expert get zeros.  x binary16 [M][K], y binary16 [M][T][N].  The rows of a
 * second product of the same experts, each with values of its own, are M T rows with T = 1.
 * Errors: INVALID_ARG (also a workspace that is too small), UNSUPPORTED, MISALIGNED, HIP. */
int w4a16_experts_gemm(const uint16_t* x, const int32_t* qweight, const uint16_t* scales, const int32_t* qzeros,
                       const int32_t* g_idx, int group_size, const int32_t* index, int M, int T, int E, int N, int K,
                       uint16_t* y, void* workspace, size_t workspace_bytes, void* stream);
int w8a16_experts_gemm(const uint16_t* x, const int32_t* qweight, const uint16_t* scales, const int32_t* qzeros,
                       const int32_t* g_idx, int group_size, const int32_t* index, int M, int T, int E, int N, int K,
                       uint16_t* y, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes of w4a16_experts_backward and w8a16_experts_backward.  For T > 1, or under act
 * order, a float per slot and channel and more, 4 M T K bytes: large batches go in several calls. */
size_t w4a16_experts_backward_workspace(int M, int T, int E, int N, int K, int act_order);

/* Gradient of the rows: dx[m] = binary16(dx0[m] + sum_t W^_e^T dy[m][t]), e = index[m][t], summed
 * in fp32 and rounded once.  dy binary16 [M][T][N] (rows of slots without an expert are not
 * read); dx0 binary16 [M][K] is a gradient that already reaches x, of a second product of the
 * same rows for instance, or NULL: 0; dx may be dx0.  Errors as w4a16_experts_gemm. */
int w4a16_experts_backward(const uint16_t* dy, const int32_t* qweight, const uint16_t* scales, const int32_t* qzeros,
                           const int32_t* g_idx, int group_size, const int32_t* index, const uint16_t* dx0, int M, int T,
                           int E, int N, int K, uint16_t* dx, void* workspace, size_t workspace_bytes, void* stream);
int w8a16_experts_backward(const uint16_t* dy, const int32_t* qweight, const uint16_t* scales, const int32_t* qzeros,
                           const int32_t* g_idx, int group_size, const int32_t* index, const uint16_t* dx0, int M, int T,
                           int E, int N, int K, uint16_t* dx, void* workspace, size_t workspace_bytes, void* stream);

/* The same for the layer itself (one expert, every row): dx = binary16(dx0 + dy W^), the
 * gradient of w4a16_gemm / w8a16_gemm.  g_idx int32 [K] or NULL.  Workspace:
 * w4a16_experts_backward_workspace(M, 1, 1, N, K, act_order). */
int w4a16_gemm_backward(const uint16_t* dy, const int32_t* qweight, const uint16_t* scales, const int32_t* qzeros,
                        const int32_t* g_idx, int group_size, const uint16_t* dx0, int M, int N, int K, uint16_t* dx,
                        void* workspace, size_t workspace_bytes, void* stream);
int w8a16_gemm_backward(const uint16_t* dy, const int32_t* qweight, const uint16_t* scales, const int32_t* qzeros,
                        const int32_t* g_idx, int group_size, const uint16_t* dx0, int M, int N, int K, uint16_t* dx,
                        void* workspace, size_t workspace_bytes, void* stream);

/* out[m] = binary16(sum_t weights[m][t] y[m][t]), fp32 sums.  y binary16 [M][T][N], N % 8 == 0,
 * out binary16 [M][N]; M N < 2^34.  Errors: INVALID_ARG, UNSUPPORTED, MISALIGNED, HIP. */
int w4a16_experts_combine(const uint16_t* y, const float* weights, int M, int T, int N, uint16_t* out, void* stream);

/* Its gradients for dout binary16 [M][N]: dy[m][t] = binary16(weights[m][t] dout[m]), dweights[m][t]
 * = sum_n dout[m][n] y[m][t][n] in fp32.  dy binary16 [M][T][N], dweights float [M][T].  M <= 2^23.
 * Errors as w4a16_experts_combine. */
int w4a16_experts_combine_backward(const uint16_t* dout, const uint16_t* y, const float* weights, int M, int T, int N,
                                   uint16_t* dy, float* dweights, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* W4A16_EXPERTS_H */
