/*
 * w4a16_head.h -- C ABI of the softmax cross entropy over a quantised vocabulary head
 * (gfx950): the layer whose N outputs are the logits of a vocabulary, with the loss in place
 * of the logits and its gradient, in pieces of the vocabulary.  No call writes the logits.
 *
 * Part of libw4a16.so; the conventions of w4a16_experts.h apply, W^ and the workspaces' among them.
 * Shapes: M rows, K channels, a head of N rows of weights of which the first vocab (1 <=
 * vocab <= N) are the vocabulary and the rest padding that takes no part.  The layer's shapes
 * are those of w4a16.h and besides K % 64 == 0, for 8-bit weights N % 16 == 0, N <= 2^24, fewer
 * than 2^32 bytes of codes, M <= 2^27; M K < 2^31.
 *   x       binary16 [M][K];  target  int32 [M]: the row's class.  A value outside [0, vocab)
 *           (-100 by convention) is a row without a target: it costs nothing, its loss, lse and
 *           gradient are 0.
 */
#ifndef W4A16_HEAD_H
#define W4A16_HEAD_H

#include "w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Workspace bytes of w4a16_head_loss and w8a16_head_loss. */
size_t w4a16_head_loss_workspace(int M, int N, int K, int act_order);

/* l_v = W^_v x[m] in fp32, v < vocab;  lse[m] = log sum_v exp l_v;  loss[m] = lse[m] - l_target.
 * loss and lse float [M].  An infinity or a NaN in a row of x, or logits beyond fp32, make that
 * row's loss and lse infinite or NaN, and no other's.
 * Errors: INVALID_ARG (also a workspace that is too small), UNSUPPORTED, MISALIGNED, HIP. */
int w4a16_head_loss(const uint16_t* x, const int32_t* qweight, const uint16_t* scales, const int32_t* qzeros,
                    const int32_t* g_idx, int group_size, const int32_t* target, int M, int N, int K, int vocab,
                    float* loss, float* lse, void* workspace, size_t workspace_bytes, void* stream);
int w8a16_head_loss(const uint16_t* x, const int32_t* qweight, const uint16_t* scales, const int32_t* qzeros,
                    const int32_t* g_idx, int group_size, const int32_t* target, int M, int N, int K, int vocab,
                    float* loss, float* lse, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes of w4a16_head_loss_backward and w8a16_head_loss_backward. */
size_t w4a16_head_loss_backward_workspace(int M, int N, int K, int act_order);

/* dx[m] = binary16(dloss[m] (sum_v exp(l_v - lse[m]) W^_v - W^_target)) for the gradient of the
 * losses, dloss float [M] (a training program puts its loss scale there: dx is binary16); lse as
 * w4a16_head_loss gave it.  The probabilities enter the product as binary16 values times
 * 2^14, fp32 sums, one rounding at the end.  The rounding of lse, 2^-24 |lse|, is an error of every
 * probability relative to it, and so an absolute one of the target's p - 1.  dx binary16 [M][K].  Errors as w4a16_head_loss. */
int w4a16_head_loss_backward(const float* dloss, const uint16_t* x, const int32_t* qweight, const uint16_t* scales,
                             const int32_t* qzeros, const int32_t* g_idx, int group_size, const int32_t* target,
                             const float* lse, int M, int N, int K, int vocab, uint16_t* dx, void* workspace,
                             size_t workspace_bytes, void* stream);
int w8a16_head_loss_backward(const float* dloss, const uint16_t* x, const int32_t* qweight, const uint16_t* scales,
                             const int32_t* qzeros, const int32_t* g_idx, int group_size, const int32_t* target,
                             const float* lse, int M, int N, int K, int vocab, uint16_t* dx, void* workspace,
                             size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* W4A16_HEAD_H */
