/*
 * vqlinear_ffn.h -- the feed-forward block around a codebook-VQ linear layer: a forward
 * with bias, activation, gate and residual in its epilogue.
 *
 * The storage format, the element types and the conventions shared by every entry point
 * (status codes and vq_last_error, streams, ownership, 16-byte alignment of device
 * pointers, one call at a time per handle) are those stated in vqlinear.h.
 */
#ifndef VQLINEAR_FFN_H
#define VQLINEAR_FFN_H

#include "vqlinear.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations act(v), computed in fp32. */
enum {
  VQ_ACT_NONE = 0,     /* v */
  VQ_ACT_RELU = 1,     /* max(v, 0) */
  VQ_ACT_SILU = 2,     /* v / (1 + exp(-v)) */
  VQ_ACT_GELU = 3,     /* v/2 (1 + erf(v / sqrt 2)) */
  VQ_ACT_GELU_TANH = 4 /* v/2 (1 + tanh(sqrt(2/pi) (v + 0.044715 v^3))) */
};

/* fp32 logits (vq_router_forward), beside VQ_F16 and VQ_BF16. */
enum { VQ_F32 = 2 };

/* ------------------------------------------------------------------ fused epilogue */

/* y = act(x . W^T + bias) * mul + residual; every part may be absent (NULL).  Elements
 * have the handle's act_dtype. */
typedef struct {
  int32_t act;          /* VQ_ACT_* */
  const void* bias;     /* [N] */
  const void* mul;      /* [M][N], e.g. the up projection of a gated pair */
  const void* residual; /* [M][N] */
} vq_epilogue;

/* vq_linear_forward with `epi` applied to the fp32 result before its one rounding into
 * y (after the sparse correction's term, if the handle carries one); with `signs` (may be
 * NULL) vq_linear_forward_rotated.  Same kernels, paths, launches, synchronisation and
 * errors as those two; bias, mul and residual are read once, and an epilogue with act
 * VQ_ACT_NONE and no tensors gives their result bit for bit.
 * mul and residual may be y itself (each element is read before it is written); any other
 * overlap of y with an input is VQ_ERR_INVALID_ARG, as is an `act` that is not a VQ_ACT_*
 * or a NULL `epi`. */
vq_status vq_linear_forward_epilogue(vq_linear_t h, const void* x, const int8_t* signs, const vq_planes* planes,
                                     const vq_codebooks* codebooks, const void* scales, const vq_epilogue* epi,
                                     void* y, int32_t M, int32_t N, int32_t K, void* stream);

/* ------------------------------------------------------------------------- routing */

typedef struct {
  int32_t E;      /* experts, 1 .. 512 */
  int32_t k;      /* experts per token, 1 .. min(E, 32) */
  int32_t renorm; /* 1: a token's k weights add up to 1; 0: they are softmax probabilities over all E */
  int32_t max_T;  /* largest token count of a call; max_T * k < 2^31 */
} vq_router_desc;

typedef struct vq_router_s* vq_router_t;

/* Create a handle on the current device (allocates the per-block expert counts).
 * Synchronous. */
vq_status vq_router_create(const vq_router_desc* desc, vq_router_t* out);
vq_status vq_router_destroy(vq_router_t h);

/* For every token t the k experts with the largest logits, largest first, equal logits in
 * the order of their numbers:
 *   ids      int32 [T][k]
 *   weights  fp32 [T][k]: exp(l - max) / sum over all experts, or over the k chosen
 *            (renorm); a logit of +inf takes the whole weight, shared by equals
 * and the T k (token, choice) pairs in the order of their experts, those of one expert in
 * the order of tokens:
 *   offsets  int32 [E+1]: pairs of expert e are offsets[e] .. offsets[e+1] - 1
 *   rows     int32 [T*k]: the token of every pair, in that order (the `rows` of
 *            vq_experts_forward on the tokens' x)
 *   slots    int32 [T][k]: the place of pair (t, j) in that order
 * A logit of -inf or NaN is masked: its expert is never chosen.  A token with fewer than
 * k experts left has ids -1, weights 0 and slots -1 in the remaining places and no pairs
 * for them; offsets[E] counts the pairs there are, and rows from offsets[E] on is left
 * as it was.
 *   logits   [T][E], VQ_F16, VQ_BF16 or VQ_F32 (`dtype`)
 * One kernel for small T, else two, on `stream`.  T == 0 writes zero offsets. */
vq_status vq_router_forward(vq_router_t h, const void* logits, int32_t dtype, int32_t* ids, float* weights,
                            int32_t* offsets, int32_t* rows, int32_t* slots, int32_t T, void* stream);

/* out[t] = RN(sum_j weights[t][j] * y[slots[t][j]] + residual[t]): the experts' rows back to
 * their tokens, summed in fp32 in the order of j, one rounding.
 *   y         [y_rows][N], VQ_F16 or VQ_BF16 (`dtype`); N % 8 == 0, else VQ_ERR_UNSUPPORTED
 *   weights   fp32 [T][k];  slots  int32 [T][k]; a slot outside [0, y_rows) contributes
 *             nothing (its weight is not used)
 *   residual  [T][N] or NULL; may be `out`
 *   out       [T][N]; must not overlap y
 * 1 <= k <= 32.  One kernel on `stream`, on the current device. */
vq_status vq_experts_combine(const void* y, int32_t y_rows, const float* weights, const int32_t* slots,
                             const void* residual, void* out, int32_t T, int32_t k, int32_t N, int32_t dtype,
                             void* stream);

#ifdef __cplusplus
}
#endif

#endif /* VQLINEAR_FFN_H */
