/*
 * vqlinear_ffn.h -- the feed-forward block around a codebook-VQ linear layer: a forward
 * with bias, activation, gate and residual in its epilogue; the same product grouped by
 * expert over ragged row counts; and the routing that feeds it (top-k experts of every
 * token, the rows in expert order, and their weighted sum back to the tokens).
 *
 * The storage format, the element types and the conventions shared by every entry point
 * (status codes and vq_last_error, streams, ownership, 16-byte alignment of device
 * pointers, one call at a time per handle) are those stated in vqlinear.h.  Row counts
 * per expert, row orders and routing results live on the device and are never read by
 * the host, so every call here can be captured into a CUDA graph and replayed on other
 * contents.
 */
#ifndef VQLINEAR_FFN_H
#define VQLINEAR_FFN_H

#include "vqlinear.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations act(v), computed in fp32 (SiLU and the tanh form of GELU give 0 where they are below
 * |v| 2^-126). */
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
 * overlap of y with an input is VQ_ERR_INVALID_ARG (of the sparse correction's entries the first
 * is looked at: the host does not know their number), as is an `act` that is not a VQ_ACT_*
 * or a NULL `epi`. */
vq_status vq_linear_forward_epilogue(vq_linear_t h, const void* x, const int8_t* signs, const vq_planes* planes,
                                     const vq_codebooks* codebooks, const void* scales, const vq_epilogue* epi,
                                     void* y, int32_t M, int32_t N, int32_t K, void* stream);

/* ---------------------------------------------------------- products grouped by expert */

/* E weight matrices of one shape.  Expert e's planes, scales and (unless shared)
 * codebooks follow expert e-1's without padding: planes->lo is [E][N*G] and so on, each
 * in the storage format of a single layer (VQ_FMT_VQ16_RVQ: idx16 is [E][n16][N*G]);
 * cb1 is [E][entries][8], and so are cb2, cbr[t] and cb8. */
typedef struct {
  vq_linear_desc layer;     /* N, K, fmt, scale_group, act_dtype, n16, n8, mult of every expert; max_M: the
                               largest row count T of a call, all experts together; rht and corr must be 0
                               (rotate x with vq_rht_apply).  N % 8 == 0 (N % 16 == 0 with glu), else
                               VQ_ERR_UNSUPPORTED */
  int32_t E;                /* 1 .. 1024 */
  int32_t shared_codebooks; /* 1: one set of codebooks for all experts */
  int32_t glu;              /* 1: rows [0, N/2) of W are a gate, rows [N/2, N) its up projection; y has N/2 columns */
  int32_t act;              /* VQ_ACT_* */
  int32_t gather;           /* 1: calls may give `rows`; create then allocates max_M x K elements, where the
                               tensor-core kernel's calls put x in row order */
} vq_experts_desc;

typedef struct vq_experts_s* vq_experts_t;

/* Create a handle on the current device (allocates an error word and, with gather, the
 * buffer for x).  Synchronous.  On error *out is set to NULL. */
vq_status vq_experts_create(const vq_experts_desc* desc, vq_experts_t* out);

/* As vq_linear_destroy. */
vq_status vq_experts_destroy(vq_experts_t h);

/* The rows r of expert e are offsets[e] <= r < offsets[e+1], and for each of them
 *   y[r] = RN(act(x[rows[r]] . W_e^T + bias[e]))                              (glu == 0)
 *   y[r] = RN(act(x[rows[r]] . G_e^T + bias[e][:N/2]) * (x[rows[r]] . U_e^T + bias[e][N/2:]))
 * with G_e, U_e the first and second N/2 rows of W_e.
 *   x        [x_rows][K], act_dtype
 *   rows     device int32 [T], the x row of every row (desc.gather == 1), or NULL: row r reads
 *            x[r] (x_rows must then be at least T).  A value outside [0, x_rows) reads as a row of zeros.
 *   offsets  device int32 [E+1], non-decreasing, offsets[0] >= 0, offsets[E] <= T; an
 *            expert with offsets[e] == offsets[e+1] has no rows and its weights are not
 *            read.  Values are clamped into [0, T] and to at least the ones before them, so
 *            bad offsets give wrong rows but no access out of range.
 *   bias     [E][N], act_dtype, or NULL
 *   y        [T][N] (glu: [T][N/2]), act_dtype.  Rows below offsets[0] or from offsets[E]
 *            on are left as they were.  A y that overlaps an input is VQ_ERR_INVALID_ARG.
 * Accumulation is fp32.  The weights are rounded to act_dtype before the product, as
 * the single-layer paths that materialise weights do: the stage sum in fp32 (one addition, or one
 * fused multiply-add per residual stage of the ladder), times the scale, rounded to fp32 and then
 * to act_dtype.  For a given kernel (below) the result of a row does not
 * depend on the other rows, and is bit-identical from run to run.
 * Enqueues one kernel on `stream` (two where VQ_PATH_TC is given rows); nothing for T == 0. */
vq_status vq_experts_forward(vq_experts_t h, const void* x, int32_t x_rows, const int32_t* rows,
                             const int32_t* offsets, const vq_planes* planes, const vq_codebooks* codebooks,
                             const void* scales, const void* bias, void* y, int32_t T, void* stream);

/* The kernel of later forwards: VQ_PATH_GEMV (warp MMAs on weights decoded in registers;
 * tiles of 16 rows of W by up to 16 rows of an expert), VQ_PATH_TC (tcgen05 on weights decoded
 * into tensor memory; tiles of 256 rows of W by up to 256), or VQ_PATH_AUTO, which goes by T, E and
 * the layer's shape: VQ_PATH_GEMV while T rows spread over min(E, T) experts come to at most 2
 * each, or 14 where the larger tiles are fewer than the SMs (the counts themselves stay on the
 * device). */
vq_status vq_experts_set_path(vq_experts_t h, int32_t path);

/* As vq_linear_plan, for a forward of T rows (launches: with rows, if desc.gather == 1). */
vq_status vq_experts_plan(vq_experts_t h, int32_t T, vq_plan_info* out);

/* As vq_linear_check, for the waits of this handle's kernels. */
vq_status vq_experts_check(vq_experts_t h, void* stream);

/* ------------------------------------------------------------------------- routing */

typedef struct {
  int32_t E;      /* experts, 1 .. 512 */
  int32_t k;      /* experts per token, 1 .. min(E, 32) */
  int32_t renorm; /* 1: a token's k weights add up to 1; 0: they are softmax probabilities over all E */
  int32_t max_T;  /* largest token count of a call, 1 .. 2^30; max_T * k < 2^31 */
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
 * logits and the five outputs must not overlap one another.
 * One kernel for small T, else two, on `stream`.  T == 0 writes zero offsets. */
vq_status vq_router_forward(vq_router_t h, const void* logits, int32_t dtype, int32_t* ids, float* weights,
                            int32_t* offsets, int32_t* rows, int32_t* slots, int32_t T, void* stream);

/* out[t] = RN(sum_j weights[t][j] * y[slots[t][j]] + residual[t]): the experts' rows back to
 * their tokens, summed in fp32 in the order of j, one rounding.
 *   y         [y_rows][N], VQ_F16 or VQ_BF16 (`dtype`); N % 8 == 0 and N <= 2^24, else VQ_ERR_UNSUPPORTED
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
