/*
 * cp_ops.h -- C ABI of the feed-forward operators that stand beside the GEMM
 * chain (cp_chain.h) on one AMD Instinct MI355X (gfx950): linear layers with
 * a fused epilogue, linear layers grouped by expert, and layer normalisation,
 * each with its backward pass.
 *
 * Conventions common to every entry point:
 *   - status codes, element types and the first two activation codes are those
 *     of cp_chain.h; no C++ exception crosses the ABI; cp_ops_last_error()
 *     gives a thread-local detail string of the calling thread's last failure;
 *   - every pointer is a DEVICE pointer owned by the caller; nothing is kept
 *     past the call, no memory is allocated and nothing is synchronised: the
 *     call enqueues kernels on `stream` (a hipStream_t, NULL = the default
 *     stream) and returns, so it may be captured into a hipGraph;
 *   - matrices are row-major with unit stride within a row and `ld` elements
 *     from one row to the next (ld >= the row's length; not read where there
 *     is at most one row).  No alignment beyond the element's own is needed;
 *     16-byte aligned rows are faster (others are copied first, see
 *     cp_ops_workspace);
 *   - sums run in fp32 (products on the matrix cores), outputs are rounded
 *     once, to nearest even, and results do not depend on timing: the same
 *     call gives the same bits;
 *   - `ws` is scratch memory of at least cp_ops_workspace() bytes, 256-byte
 *     aligned, with any contents; calls that may overlap need their own;
 *   - an output shares no memory with an input or another output unless
 *     stated; Y and pre that do are refused with CP_ERR_INVALID_ARG (rows of
 *     one buffer may interleave);
 *   - sizes of zero are allowed unless stated: empty outputs are left alone,
 *     a sum over nothing is zero.
 */
#ifndef CP_OPS_H
#define CP_OPS_H

#include <stdint.h>

#include "cp_chain.h"

#ifdef __cplusplus
extern "C" {
#endif

/* activations of the operators, besides CP_ACT_NONE and CP_ACT_GELU_TANH */
#define CP_ACT_RELU 2 /* max(x, 0), derivative 0 at 0; NaN stays NaN */
#define CP_ACT_SILU 3 /* x / (1 + exp(-x))        */

/* operator codes of cp_ops_workspace */
#define CP_OP_LINEAR 0
#define CP_OP_LINEAR_BACKWARD 1
#define CP_OP_GROUPED_LINEAR 2
#define CP_OP_GROUPED_LINEAR_BACKWARD 3
#define CP_OP_LAYER_NORM_BACKWARD 4

/* rows, columns and leading dimensions are at most this many elements (rows
 * of the activations: 2^30), and an operator takes at most CP_OPS_MAX_GROUPS
 * experts.  A product whose result has 2^23 tiles of 256 x 256 or more (fp32:
 * 2^24 of 128 x 128; with at most 16 rows per expert: 2^24 of 16 x 128, an
 * expert's last one counting in full) is refused with CP_ERR_SHAPE. */
#define CP_OPS_MAX_WIDTH 4194304
#define CP_OPS_MAX_GROUPS 4096

/*
 * cp_linear -- Y = act(X W + b) + R, and the pre-activation X W + b if `pre`
 * is given.
 *   X[M][K], W[K][N] (w_trans = 0) or stored as [N][K] (w_trans = 1),
 *   bias[N] or NULL, R[M][N] or NULL, Y[M][N], pre[M][N] or NULL
 * Y may be R (same pointer and ld).
 */
int cp_linear(int32_t dtype, int64_t M, int64_t K, int64_t N, const void *X, int64_t ldx, const void *W, int64_t ldw,
              int32_t w_trans, const void *bias, const void *R, int64_t ldr, int32_t act, void *Y, int64_t ldy,
              void *pre, int64_t ldp, void *ws, int64_t ws_bytes, void *stream);

/*
 * cp_linear_backward -- gradients of cp_linear for dY[M][N]:
 *   dZ = dY act'(pre)   dX = dZ W^t   dW = X^t dZ   db = sum over rows of dZ
 * (the gradient of R is dY itself).  `pre` is what cp_linear stored; it may be
 * NULL only with CP_ACT_NONE.  dX, dW and db may each be NULL; dW has W's
 * layout (w_trans).  X may be NULL without dW, W without dX.  With bf16 and
 * an activation, dZ is rounded to bf16 before the two products (they run on
 * the bf16 matrix cores); db sums the unrounded dZ.
 */
int cp_linear_backward(int32_t dtype, int64_t M, int64_t K, int64_t N, const void *dY, int64_t lddy, const void *X,
                       int64_t ldx, const void *W, int64_t ldw, int32_t w_trans, const void *pre, int64_t ldp,
                       int32_t act, void *dX, int64_t lddx, void *dW, int64_t lddw, void *db, void *ws,
                       int64_t ws_bytes, void *stream);

/*
 * cp_grouped_linear -- rows sorted by expert, each through its expert's layer:
 *   Y[t] = act(X[t] W_e + b_e)   for offsets[e] <= t < offsets[e + 1]
 *   X[T][K], Y[T][N], pre[T][N] or NULL; W_e at W + e * stride_w, each as in
 *   cp_linear; bias[E][N] or NULL; offsets[E + 1]: int32, DEVICE memory
 * The host never reads the offsets.  They are meant to start at 0 and not to
 * decrease; the device takes the first as 0 and each as the largest so far,
 * between 0 and T, so that no value reads or writes out of range.  Rows from
 * offsets[E] on belong to no expert: their Y and pre are zero.  1 <= E <= CP_OPS_MAX_GROUPS.
 */
int cp_grouped_linear(int32_t dtype, int64_t T, int64_t K, int64_t N, int32_t E, const void *X, int64_t ldx,
                      const void *W, int64_t ldw, int64_t stride_w, int32_t w_trans, const int32_t *offsets,
                      const void *bias, int32_t act, void *Y, int64_t ldy, void *pre, int64_t ldp, void *ws,
                      int64_t ws_bytes, void *stream);

/*
 * cp_grouped_linear_backward -- its gradients, as cp_linear_backward per
 * expert.  dW[E] (layout of W, expert e at dW + e * stride_dw) and db[E][N]
 * are zero for experts without rows; dX is zero for rows without an expert.
 */
int cp_grouped_linear_backward(int32_t dtype, int64_t T, int64_t K, int64_t N, int32_t E, const void *dY, int64_t lddy,
                               const void *X, int64_t ldx, const void *W, int64_t ldw, int64_t stride_w,
                               int32_t w_trans, const int32_t *offsets, const void *pre, int64_t ldp, int32_t act,
                               void *dX, int64_t lddx, void *dW, int64_t lddw, int64_t stride_dw, void *db, void *ws,
                               int64_t ws_bytes, void *stream);

/*
 * cp_layer_norm -- Y = (X - mean) rstd w + b per row, rstd = 1 / sqrt(var +
 * eps) with var the mean squared deviation.  w[N] and b[N] may each be NULL
 * (ones, zeros); mean[M] and rstd[M], fp32, may each be NULL.  N >= 1 (where
 * M >= 1), eps >= 0.  Y may be X (same pointer and ld).
 */
int cp_layer_norm(int32_t dtype, int64_t M, int64_t N, const void *X, int64_t ldx, const void *w, const void *b,
                  float eps, void *Y, int64_t ldy, float *mean, float *rstd, void *stream);

/*
 * cp_layer_norm_backward -- with xh = (X - mean) rstd and g = dY w:
 *   dX = rstd (g - mean(g) - xh mean(g xh))   dw = sum over rows of dY xh
 *   db = sum over rows of dY
 * w may be NULL (ones); dX, dw and db may each be NULL.  dX may be dY or X
 * (same pointer and ld).
 */
int cp_layer_norm_backward(int32_t dtype, int64_t M, int64_t N, const void *dY, int64_t lddy, const void *X,
                           int64_t ldx, const float *mean, const float *rstd, const void *w, void *dX, int64_t lddx,
                           void *dw, void *db, void *ws, int64_t ws_bytes, void *stream);

/*
 * cp_ops_workspace -- bytes of scratch memory the operator `op` (CP_OP_*)
 * needs at these sizes, whatever its optional arguments; may be 0.  K is
 * ignored by CP_OP_LAYER_NORM_BACKWARD, E by the dense operators.  `aligned`:
 * X, W and dY have 16-byte aligned pointers, row strides, expert strides and
 * row lengths; without that (0) there is room for copies of them that do.
 * Negative status code on bad arguments.  Host only, no device needed.
 */
int64_t cp_ops_workspace(int32_t op, int32_t dtype, int64_t M, int64_t K, int64_t N, int32_t E, int32_t aligned);

/* cp_ops_last_error -- thread-local detail of the calling thread's most recent
 * failure in this header's functions ("" if its last call succeeded). */
const char *cp_ops_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* CP_OPS_H */
