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

#ifdef __cplusplus
}
#endif

#endif /* VQLINEAR_FFN_H */
