/*
 * cp_ops.h -- C ABI of the feed-forward operators that stand beside the GEMM
 * chain (cp_chain.h) on one AMD Instinct MI355X (gfx950): linear layers with
 * a fused epilogue, linear layers grouped by expert, layer normalisation, the
 * router of an expert layer and its rows' way to the experts and back, each
 * with its backward pass; linear layers with 4-bit weights; the gradients'
 * norm and clipping.
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
#define CP_OP_ROUTE 5          /* M: tokens, N: experts */
#define CP_OP_CLIP_GRAD_NORM 6 /* M: tensors            */
#define CP_OP_LINEAR_INT4 7    /* E = 0: dense          */

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

/* experts that cp_route chooses from, experts to a token, and tensors of
 * cp_clip_grad_norm, at most */
#define CP_OPS_MAX_ROUTED 1024
#define CP_OPS_MAX_CHOSEN 32
#define CP_OPS_MAX_TENSORS 16777216

/*
 * cp_route -- the router of an expert layer: of each token's logits[T][E]
 *   p = softmax(logits)
 *   experts[T][k]  the k largest, largest first, the lower index of equals; -1
 *                  where no expert is left (a logit of -inf is never chosen)
 *   gates[T][k]    fp32: p of the chosen; with `normalize` divided by their
 *                  sum; 0 for slots without an expert
 *   counts[E]      slots of each expert
 *   offsets[E + 1] their running sum, as cp_grouped_linear takes it
 *   rows[T][k]     each slot's row among the offsets[E] rows sorted by expert
 *                  and, within an expert, by token; -1 for slots without one
 *   loss           fp32, the balance loss E sum_e f_e P_e with f_e = counts_e /
 *                  (n k) and P_e = sum_t p_te / n over the n tokens that have
 *                  an expert; 0 without any
 *   slopes[E]      fp32, d loss / d p_te (counts being constants): E counts_e /
 *                  (n^2 k)
 * valid[T], one byte each, or NULL: tokens with 0 are padding and have no
 * expert.  NaN counts as the largest logit; a row that holds NaN or +inf has
 * gates of NaN, as a softmax has.  1 <= E <= CP_OPS_MAX_ROUTED, 1 <= k <= E and
 * CP_OPS_MAX_CHOSEN, T k <= 2^30.  All vectors are contiguous.
 */
int cp_route(int32_t dtype, int64_t T, int32_t E, int32_t k, int32_t normalize, const void *logits, int64_t ld,
             const uint8_t *valid, int32_t *experts, float *gates, int32_t *rows, int32_t *counts, int32_t *offsets,
             float *loss, float *slopes, void *ws, int64_t ws_bytes, void *stream);

/*
 * cp_route_backward -- dlogits[T][E] of cp_route for dgates[T][k] and dloss
 * (fp32, device memory; each may be NULL: zero), from the same logits and the
 * experts and slopes it gave (a token's experts are different).  Counts are
 * constants.  Zero for tokens without an expert.  dlogits may be logits (same pointer and ld).
 */
int cp_route_backward(int32_t dtype, int64_t T, int32_t E, int32_t k, int32_t normalize, const float *dgates,
                      const float *dloss, const void *logits, int64_t ld, const int32_t *experts, const float *slopes,
                      void *dlogits, int64_t ldd, void *stream);

/*
 * cp_dispatch -- tokens' rows to their experts: out[rows[t][j]] = x[t] for
 * x[T][D], out[R][D].  Rows of `out` from *end on (device memory, offsets[E] of
 * cp_route) are zero.  Entries of rows[T][k] outside 0 .. R - 1 are no slots;
 * the others are meant to be different.  Rows that no slot names and that lie
 * before *end are left as they were.  Its gradient is cp_combine without gates.
 */
int cp_dispatch(int32_t dtype, int64_t T, int32_t k, int64_t R, int64_t D, const void *x, int64_t ldx,
                const int32_t *rows, const int32_t *end, void *out, int64_t ldo, void *stream);

/*
 * cp_combine -- experts' rows back to their tokens:
 *   out[t] = sum_j gates[t][j] y[rows[t][j]] + res[t]
 * y[R][D], gates[T][k] fp32 or NULL (ones), res[T][D] or NULL, out[T][D].
 * Slots are added in order, in fp32; those that are none (see cp_dispatch) are
 * left out, their gates are not read into the sum.  out may be res (same
 * pointer and ld).
 */
int cp_combine(int32_t dtype, int64_t T, int32_t k, int64_t R, int64_t D, const void *y, int64_t ldy,
               const int32_t *rows, const float *gates, const void *res, int64_t ldr, void *out, int64_t ldo,
               void *stream);

/*
 * cp_combine_backward -- its gradients for dout[T][D]:
 *   dy[rows[t][j]] = gates[t][j] dout[t], zero from *end on
 *   dgates[t][j]   = sum_d dout[t][d] y[rows[t][j]][d], fp32, 0 without a slot
 * dy[R][D] and dgates[T][k] may each be NULL; y may be NULL without dgates,
 * end without dy.  (The gradient of res is dout itself.)  The order in which a
 * token's dgates are added up goes by T, k and D, so with other tokens in the call
 * they may differ in the last bits.
 */
int cp_combine_backward(int32_t dtype, int64_t T, int32_t k, int64_t R, int64_t D, const void *dout, int64_t ldd,
                        const void *y, int64_t ldy, const int32_t *rows, const int32_t *end, const float *gates,
                        void *dy, int64_t lddy, float *dgates, void *stream);

/*
 * 4-bit weights: w[k][n] = scales[k / group][n] (codes[k][n] - zeros[k / group][n])
 * with codes and zero points of 0 .. 15 in a byte each (higher bits are not
 * read); without zero points they are 8.  `group` is 32, 64 or a multiple of
 * 128, a last group may be shorter; there are ceil(K / group) of them.  dtype is
 * that of the scales and of the rows the layer takes.  E >= 1 experts, one
 * after another.
 *
 * cp_int4_quantize -- codes[E][K][N], scales[E][groups][N] and zeros[E][groups][N]
 * (or NULL: symmetric, 7 steps to either side) of a finite weight, whose element
 * (e, k, n) is at W + e stride_e + k stride_k + n stride_n elements.
 * cp_int4_pack -- lays codes, scales and zero points (or NULL), contiguous, out
 * for cp_linear_int4, in cp_int4_bytes() bytes at `packed`, 16-byte aligned.
 * cp_int4_bytes is host only; a negative status code on bad arguments.
 */
int cp_int4_quantize(int32_t dtype, int64_t K, int64_t N, int32_t E, int64_t group, const void *W, int64_t stride_k,
                     int64_t stride_n, int64_t stride_e, uint8_t *codes, void *scales, uint8_t *zeros, void *stream);
int64_t cp_int4_bytes(int32_t dtype, int64_t K, int64_t N, int32_t E, int64_t group);
int cp_int4_pack(int32_t dtype, int64_t K, int64_t N, int32_t E, int64_t group, const uint8_t *codes,
                 const void *scales, const uint8_t *zeros, void *packed, void *stream);

/*
 * cp_linear_int4, cp_grouped_linear_int4 -- cp_linear and cp_grouped_linear with
 * a packed weight, for decoding and short prompts: the layer with a bf16 weight is
 * faster from about 400 rows on, from about 100 where that weight stays in the last
 * cache (8192 x 8192: 256 rows 56 us, with bf16 63 and in the cache 45; 2048 rows
 * 433 to 454 and 195 to 208).
 * Products of x with the codes are exact and added up in fp32, a group at a time;
 * the weight itself is never rounded.  With fp32 rows a result is as good as that of
 * the weight in fp32; with bf16 rows it is off by a few 2^-24 of 31 scales sum |x|
 * beside its rounding to bf16, also where all codes are their zero points.  x is
 * meant to be finite and below 2^115: a
 * row with infinities gives NaN.  More than 2^22 workgroups are refused with
 * CP_ERR_SHAPE: tiles of 32 x 64 at least (an expert's last one counting in full)
 * or, with at most 16 rows to an expert, experts times parts of K of 2048 at least.
 */
int cp_linear_int4(int32_t dtype, int64_t M, int64_t K, int64_t N, const void *X, int64_t ldx, const void *packed,
                   int64_t group, const void *bias, const void *R, int64_t ldr, int32_t act,
                   void *Y, int64_t ldy, void *ws, int64_t ws_bytes, void *stream);
int cp_grouped_linear_int4(int32_t dtype, int64_t T, int64_t K, int64_t N, int32_t E, const void *X, int64_t ldx,
                           const void *packed, int64_t group, const int32_t *offsets,
                           const void *bias, int32_t act, void *Y, int64_t ldy, void *ws, int64_t ws_bytes,
                           void *stream);

/*
 * cp_clip_grad_norm -- norm = sqrt(sum of squares over all of n tensors), added up
 * in fp64, and outs[i] = grads[i] min(1, max_norm / (norm + 1e-6)).
 *   dtypes[n], grads[n], numels[n], out_dtypes[n], outs[n]: HOST arrays, read
 *   during the call; tensor i has numels[i] elements side by side, all together
 *   2^44 at most
 * outs[i] may be grads[i] (of the same type); apart from that no output, norm among
 * them, shares memory with an input or another output, which is checked.  outs NULL:
 * the norm alone (out_dtypes is not read).  norm: fp32, device memory.  max_norm >= 0;
 * with an infinite one nothing is scaled; a norm that is not finite makes the factor
 * 0 or NaN.  n may be 0: the norm is 0.
 */
int cp_clip_grad_norm(int64_t n, const int32_t *dtypes, const void *const *grads, const int64_t *numels,
                      float max_norm, const int32_t *out_dtypes, void *const *outs, float *norm, void *ws,
                      int64_t ws_bytes, void *stream);

/*
 * cp_ops_workspace -- bytes of scratch memory the operator `op` (CP_OP_*)
 * needs at these sizes, whatever its optional arguments; may be 0.  K is
 * ignored by CP_OP_LAYER_NORM_BACKWARD and the two codes after it, E by the
 * dense operators and those.  `aligned`:
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
