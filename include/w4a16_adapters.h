/*
 * w4a16_adapters.h -- C ABI of the low-rank adapters beside the quantised layer, their
 * gradients, and the layer's input kept in 8 bits for the backward pass (gfx950).
 *
 * The layer's weights are frozen in 4 or 8 bits; what is served per request and what is
 * trained are low-rank adapters added to its output: y + s B (A x) with A [R][K] and B
 * [N][R].  One call takes the rows of many requests, each with an adapter of its own.
 * Part of libw4a16.so; statuses, w4a16_last_error and the conventions of w4a16.h apply:
 * device pointers, everything asynchronous and ordered on `stream`, the stream belongs to
 * the current device, no exception crosses the ABI, nothing is launched on failure.
 *
 * Shapes: M rows, K input and N output channels, rank R, L adapters; M, K, N > 0,
 * K % 8 == 0, N % 8 == 0, R % 8 == 0, 8 <= R <= 128 (pad a smaller rank with zeros),
 * 1 <= L <= 65535, M <= 2^27, N and K <= 2^24.  Sizes whose launches would pass 2^32 threads
 * are refused as well: the gradients of L adapters from L (N + K) of about 2^30 on (half of it
 * for a rank above 32, and so on per 32 ranks), and rows and channels that no device holds.
 *   x, y, out       binary16 [M][K], [M][N], [M][N], row-major
 *   a               binary16 [L][R][K];  b  binary16 [L][N][R]
 *   index           int32 [M], adapter of every row, or NULL: adapter 0 for every row.  A
 *                   value outside [0, L) (-1 by convention) is a row without an adapter.
 *                   Rows may come in any order.  Grouping them (more than 256 rows, or a
 *                   backward pass) reads the index twice per adapter.
 *   scaling         float [L] (alpha / rank of every adapter) or NULL: 1
 *   h               float [M][R], A_i x of every row, 0 for rows without an adapter
 *   workspace       16-byte aligned device memory of at least the size that the matching
 *                   _workspace function returns for the same sizes, owned by the caller
 *                   and free again once the stream has passed the call.  No call
 *                   allocates, so every call can be captured into a graph; two graphs (or
 *                   streams) that may run at once need a workspace each.
 * Buffers must be 16-byte aligned (index and scaling: 4-byte aligned).  Outputs must not
 * overlap inputs or the workspace, but for the two pairs named below.  Results do not
 * depend on timing: every sum has a fixed order.  Sums of products are fp32 sums, except that
 * an operand x, a, b or dy below 2^-14 (subnormal) counts as 2^-14 in their rounding errors.
 * An infinity or a NaN in an operand makes the results that it enters infinite or NaN (not
 * always which of the two the formula gives), and no others: rows keep to themselves,
 * gradients to their adapter.
 */
#ifndef W4A16_ADAPTERS_H
#define W4A16_ADAPTERS_H

#include "w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Workspace bytes of w4a16_lora_forward: 0 where the call needs none (workspace may then be
 * NULL), and on sizes that it refuses.  with_index: 1 when index is not NULL. */
size_t w4a16_lora_forward_workspace(int M, int N, int K, int R, int L, int with_index);

/* out[m] = binary16(y[m] + s_i B_i (A_i x[m])), i = index[m]: binary16 operands, fp32 sums,
 * A_i x within 2^-23 of itself between the two products, one rounding at the end.  Rows without an
 * adapter: out[m] = y[m], bit for bit.  out may be y (in place).  h: NULL, or where A_i x
 * is written for the backward pass.
 * Errors: INVALID_ARG (also a workspace that is too small), UNSUPPORTED (R, L, sizes),
 * MISALIGNED, HIP. */
int w4a16_lora_forward(const uint16_t* y, const uint16_t* x, const uint16_t* a, const uint16_t* b,
                       const int32_t* index, const float* scaling, int M, int N, int K, int R, int L,
                       uint16_t* out, float* h, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes of w4a16_lora_backward and w4a16_lora_backward_q8; 0 on refused sizes. */
size_t w4a16_lora_backward_workspace(int M, int N, int K, int R, int L, int with_index);

/* Gradients of w4a16_lora_forward for the output gradient dy binary16 [M][N], with
 * g[m] = B_i^T dy[m] (fp32; every g and h enters the products within 2^-23 of itself, however
 * far rows and ranks lie apart):
 *   da float [L][R][K]: da_i = s_i sum g[m] x[m]^T,   db float [L][N][R]: db_i = s_i sum
 *   dy[m] h[m]^T, over the rows with index i (zeros for an adapter without rows);
 *   dx binary16 [M][K]: dx[m] = binary16(dx0[m] + s_i A_i^T g[m]); rows without an adapter
 *   keep dx0.
 * x and h as in the forward call.  dx0 binary16 [M][K] is the gradient that reaches x
 * through the quantised weights (dy W^, for which w4a16_dequant gives W^) or NULL: 0; dx
 * may be dx0.  dx NULL: not computed (dx0 is then NULL too).  da and db are overwritten.
 * Errors as w4a16_lora_forward. */
int w4a16_lora_backward(const uint16_t* dy, const uint16_t* x, const uint16_t* a, const uint16_t* b,
                        const float* h, const int32_t* index, const float* scaling, const uint16_t* dx0,
                        int M, int N, int K, int R, int L, uint16_t* dx, float* da, float* db,
                        void* workspace, size_t workspace_bytes, void* stream);

/* The same from a checkpoint of x in 8 bits (w4a16_act_quantize): x[m][k] is the value that
 * w4a16_act_dequantize restores, expanded in registers.  Bit-identical to
 * w4a16_lora_backward on the restored x.  group_size in {32, 64, 128}, K % group_size == 0,
 * M K < 2^34.
 * codes are 8-byte aligned, scales 2-byte aligned. */
int w4a16_lora_backward_q8(const uint16_t* dy, const uint8_t* codes, const uint16_t* scales, int group_size,
                           const uint16_t* a, const uint16_t* b, const float* h, const int32_t* index,
                           const float* scaling, const uint16_t* dx0, int M, int N, int K, int R, int L,
                           uint16_t* dx, float* da, float* db, void* workspace, size_t workspace_bytes,
                           void* stream);

/* Activations in 8 bits, one binary16 scale per row and group of group_size channels
 * ("LLM Quantization: INT8, GPTQ, and AWQ Explained", What quantization actually does: the
 * absmax scheme):
 *   a = max |x| of the group,  S = smallest binary16 >= a / 127 (1 if a == 0; 515.5, the
 *   largest S whose 127-fold is a binary16, for a above 127 * 515.5)
 *   codes = clamp(round(x / S), -127, 127) + 128, round half to even
 * A group that holds an infinity or a NaN gets S = NaN, so its restored values are NaN.
 *   x binary16 [M][K];  codes out uint8 [M][K];  scales out binary16 [M][K / group_size]
 * group_size in {32, 64, 128}, K % group_size == 0, M K < 2^34.  x 16-byte, codes 8-byte, scales 2-byte
 * aligned.  Errors: INVALID_ARG, UNSUPPORTED (group_size), MISALIGNED, HIP. */
int w4a16_act_quantize(const uint16_t* x, int M, int K, int group_size, uint8_t* codes, uint16_t* scales,
                       void* stream);

/* x out binary16 [M][K]: binary16((codes - 128) * S).  Errors as w4a16_act_quantize. */
int w4a16_act_dequantize(const uint8_t* codes, const uint16_t* scales, int M, int K, int group_size,
                         uint16_t* x, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* W4A16_ADAPTERS_H */
