/*
 * signmuon_layers.h - C ABI of libsignmuon.so: layers of a transformer, forward
 * and backward, as HIP kernels for AMD Instinct MI355X (gfx950): layer norm and
 * embedding lookup, the root-mean-square norm of a residual stream, the gated
 * feed-forward block, and the softmax cross entropy of a linear output layer.
 * Their weight gradients end in the float32 gradient G of signmuon_step; like
 * every result of this library they are bit-reproducible run to run, so that
 * replicas which vote on one bit per entry start from the same gradient.
 *
 * The conventions of signmuon.h hold: device pointers, caller-owned memory
 * and workspaces, asynchronous work on the caller's stream (a stream of the
 * current device), no synchronisation, argument errors before anything is
 * enqueued, no floating-point atomics.  A call enqueues only kernels on the
 * caller's stream, so it can be captured into a HIP graph; a graph keeps the
 * pointers of its capture, and calls or graphs that may run at the same time
 * need workspaces of their own.  Unless an entry point says otherwise arrays
 * do not overlap.  Pointers are aligned to their element type; no larger
 * alignment is needed.
 *
 * Dtypes are sm_dtype codes.  Every sum is held in float32 or wider; a
 * bfloat16 result is rounded once, to nearest even, when it is stored.
 *
 * A row stride counts elements; it is at most 2^39, and times the number of rows
 * at most 2^60.
 */
#ifndef SIGNMUON_LAYERS_H
#define SIGNMUON_LAYERS_H

#include "signmuon.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Layer norm of the rows of X, rows x cols:
 *   mean_r = sum_c X[r,c] / cols,  var_r = sum_c (X[r,c] - mean_r)^2 / cols,
 *   rstd_r = 1 / sqrt(var_r + eps),
 *   Y[r,c] = (X[r,c] - mean_r) * rstd_r * gamma[c] + beta[c].
 * Row r of X starts at element r * x_stride (x_stride >= cols); Y is
 * contiguous, of X's dtype, and may be X itself if X is contiguous.  gamma,
 * beta: [cols] of w_dtype; gamma NULL stands for ones, beta NULL for zeros.
 * mean, rstd: float32[rows] outputs for the backward pass, or NULL.
 * 0 <= rows < 2^31, 1 <= cols <= 2^20, eps >= 0 and finite.  rows = 0 is a
 * no-op.  A non-finite entry makes its own row NaN and no other.  So may a row
 * whose sum is past float32; where the sum of the squared deviations is, the
 * variance counts as infinite and rstd is 0.
 */
sm_status signmuon_layer_norm(const void *X, int32_t x_dtype, int64_t x_stride,
                              const void *gamma, const void *beta,
                              int32_t w_dtype, int64_t rows, int64_t cols,
                              float eps, void *Y, float *mean, float *rstd,
                              hipStream_t stream);

/*
 * Backward pass of signmuon_layer_norm for the gradient dY of Y: with
 * xhat = (X - mean) * rstd and g = dY * gamma,
 *   dX[r,c] = rstd_r * (g - sum_c(g) / cols - xhat * sum_c(g xhat) / cols),
 *   dgamma[c] = sum_r dY[r,c] xhat[r,c],  dbeta[c] = sum_r dY[r,c].
 * dY and X have x_dtype and row strides of their own (>= cols); mean and
 * rstd are what the forward pass wrote.  dX: contiguous, of x_dtype, and may
 * be dY itself if that is contiguous.  dgamma, dbeta: [cols] of dw_dtype.
 * Each of dX, dgamma and dbeta may be NULL: it is not computed then.
 * accumulate = 1 adds dgamma and dbeta to what is there (float32 only);
 * 0 overwrites it.  rows = 0 gives sums of nothing: zeros (or, when
 * accumulating, no change).  Limits as for signmuon_layer_norm.
 * ws: signmuon_layer_norm_backward_workspace() bytes, 256-byte aligned;
 * NULL where that is 0.  Its contents on entry do not matter.  The query
 * returns SIZE_MAX for rows or cols outside the limits.
 */
size_t signmuon_layer_norm_backward_workspace(int64_t rows, int64_t cols);
sm_status signmuon_layer_norm_backward(
    const void *dY, int64_t dy_stride, const void *X, int32_t x_dtype,
    int64_t x_stride, const void *gamma, int32_t w_dtype, const float *mean,
    const float *rstd, int64_t rows, int64_t cols, void *dX, void *dgamma,
    void *dbeta, int32_t dw_dtype, int32_t accumulate, void *ws,
    size_t ws_bytes, hipStream_t stream);

/*
 * Embedding lookup: Y[i,:] = scale * W[tokens[i],:] for i < n.  W:
 * contiguous vocab x dim of w_dtype; Y: contiguous n x dim of y_dtype.
 * tokens: n integers of token_bits (32 or 64) bits.  A token outside
 * [0, vocab) reads nothing and makes its row NaN, which the optimizer step
 * reports as a non-finite gradient.  0 <= n <= 2^30, 1 <= vocab, dim <= 2^20,
 * scale finite.  n = 0 is a no-op.
 */
sm_status signmuon_embedding(const void *W, int32_t w_dtype, int64_t vocab,
                             int64_t dim, const void *tokens,
                             int32_t token_bits, int64_t n, float scale,
                             void *Y, int32_t y_dtype, hipStream_t stream);

/*
 * Gradient of the embedding table: dW[v,:] = scale * sum of dY[i,:] over the
 * i < n with tokens[i] = v, for every v < vocab (zeros where there is none);
 * accumulate = 1 (float32 only) adds that to dW instead and leaves the other
 * rows untouched.  Tokens equal to padding (-1: none) and tokens outside
 * [0, vocab) add nothing.  Row i of dY starts at element i * dy_stride
 * (dy_stride >= dim).  The rows of one token are added in an order that n
 * and the tokens alone decide.  n <= 2^27, other limits as for
 * signmuon_embedding; padding is -1 or in [0, vocab).
 * ws: signmuon_embedding_backward_workspace() bytes, 256-byte aligned; NULL
 * where that is 0 (small batches).  Its contents on entry do not matter.  The
 * query returns SIZE_MAX for arguments outside the limits.
 */
size_t signmuon_embedding_backward_workspace(int64_t n, int64_t vocab,
                                             int64_t dim);
sm_status signmuon_embedding_backward(
    const void *dY, int32_t dy_dtype, int64_t dy_stride, const void *tokens,
    int32_t token_bits, int64_t n, int64_t padding, float scale, void *dW,
    int32_t dw_dtype, int64_t vocab, int64_t dim, int32_t accumulate, void *ws,
    size_t ws_bytes, hipStream_t stream);

/*
 * Root-mean-square norm of a residual stream's rows, rows x cols:
 *   H = X + R (rounded to x_dtype; H = X where R is NULL),
 *   rstd_r = 1 / sqrt(sum_c H[r,c]^2 / cols + eps),
 *   Y[r,c] = H[r,c] * rstd_r * gamma[c].
 * X, R and H have x_dtype; X and R row strides of their own (>= cols), H and Y
 * are contiguous.  H is written where R is given (and may be X or R itself if
 * that is contiguous), and is ignored otherwise; Y may be X itself if that is
 * contiguous (then H is not X).  gamma: [cols] of w_dtype, NULL for ones.
 * rstd: float32[rows] for the backward pass, or NULL.  0 <= rows < 2^31,
 * 1 <= cols <= 2^20, eps >= 0 and finite.  rows = 0 is a no-op.  A row with a NaN
 * is NaN; where the sum of the squares is past float32, rstd is 0.
 *
 * signmuon_rms_norm_e4m3 writes Y in 8 bits: row r is cut into blocks of `block`
 * = 128 columns (the last may be shorter), or is one block where block is 0;
 *   scales[r,b] = max(max |Y| of the block / 448, 2^-126),
 *   Q[r,c] = Y[r,c] / scales[r,b] to the nearest e4m3 value (OCP, no infinities).
 * Q: rows x cols bytes; scales: float32, rows x number of blocks.  cols <= 16384.
 */
sm_status signmuon_rms_norm(const void *X, int64_t x_stride, const void *R,
                            int64_t r_stride, int32_t x_dtype,
                            const void *gamma, int32_t w_dtype, int64_t rows,
                            int64_t cols, float eps, void *H, void *Y,
                            float *rstd, hipStream_t stream);
sm_status signmuon_rms_norm_e4m3(const void *X, int64_t x_stride,
                                 const void *R, int64_t r_stride,
                                 int32_t x_dtype, const void *gamma,
                                 int32_t w_dtype, int64_t rows, int64_t cols,
                                 float eps, int64_t block, void *H, void *Q,
                                 float *scales, float *rstd,
                                 hipStream_t stream);

/*
 * Backward pass of signmuon_rms_norm for the gradients dY of Y and dH of H (NULL
 * for zeros): with xhat = H * rstd and g = dY * gamma,
 *   dX[r,c] = dH[r,c] + rstd_r * (g - xhat * sum_c(g xhat) / cols),
 *   dgamma[c] = sum_r dY[r,c] xhat[r,c];
 * dX is the gradient of X and of R.  dY, H and dH have x_dtype and row strides of
 * their own (>= cols); dX: contiguous, of x_dtype, and may be dY or dH itself if
 * that is contiguous.  dgamma: [cols] of dw_dtype.  Either may be NULL: it is not
 * computed then.  accumulate = 1 adds dgamma to what is there (float32 only).
 * rows = 0 gives sums of nothing.  Workspace as for signmuon_layer_norm_backward.
 */
size_t signmuon_rms_norm_backward_workspace(int64_t rows, int64_t cols);
sm_status signmuon_rms_norm_backward(
    const void *dY, int64_t dy_stride, const void *H, int64_t h_stride,
    const void *dH, int64_t dh_stride, int32_t x_dtype, const void *gamma,
    int32_t w_dtype, const float *rstd, int64_t rows, int64_t cols, void *dX,
    void *dgamma, int32_t dw_dtype, int32_t accumulate, void *ws,
    size_t ws_bytes, hipStream_t stream);

/*
 * Gated feed-forward block of the rows of X, rows x dim:
 *   gate = X Wg^T, up = X Wu^T,  Y = (act(gate) * up) Wd^T,
 * act: SM_ACT_SILU, x / (1 + exp(-x)), or SM_ACT_GELU, x Phi(x).  Wg, Wu:
 * contiguous hidden x dim; Wd: contiguous dim x hidden; Y: contiguous rows x dim;
 * all of `dtype`.  Row r of X starts at element r * x_stride (x_stride >= dim).
 * pre: float32[rows x 2 hidden], gate and then up of a row, for the backward pass,
 * or NULL.  0 <= rows <= 2^22, 1 <= dim, hidden <= 2^16.  rows = 0 is a no-op.
 * What lies between the products is rounded to `dtype` once; in bfloat16, where
 * rows times the lesser of dim and hidden is below 4096, to a sum of two values.
 * Products of float32 are sums of products of bfloat16 parts, with float32's
 * precision for operands of 2^-109 and more (smaller ones are held to 2^-133); an
 * infinity among their operands makes NaN of what depends on it.
 * ws: signmuon_gated_mlp_workspace() bytes (backward = 1 for the backward call),
 * 256-byte aligned; NULL where that is 0.  Its contents on entry do not matter.
 * The query returns SIZE_MAX for arguments outside the limits.
 */
enum { SM_ACT_SILU = 0, SM_ACT_GELU = 1 };
size_t signmuon_gated_mlp_workspace(int64_t rows, int64_t dim, int64_t hidden,
                                    int32_t dtype, int32_t backward);
sm_status signmuon_gated_mlp(const void *X, int64_t x_stride, const void *Wg,
                             const void *Wu, const void *Wd, int32_t dtype,
                             int32_t act, int64_t rows, int64_t dim,
                             int64_t hidden, void *Y, float *pre, void *ws,
                             size_t ws_bytes, hipStream_t stream);

/*
 * Its backward pass for the gradient dY of Y, from what the forward pass wrote to
 * pre: with h = act(gate) * up and dh = dY Wd,
 *   dgate = dh * up * act'(gate),  dup = dh * act(gate),
 *   dX = dgate Wg + dup Wu,  dWg = dgate^T X,  dWu = dup^T X,  dWd = dY^T h.
 * dY has a row stride of its own (>= dim).  dX: contiguous, of `dtype`; dWg, dWu,
 * dWd: contiguous, of dw_dtype; accumulate = 1 adds to what is there (float32
 * only).  Each may be NULL: it is not computed then.  rows = 0 gives sums of
 * nothing.
 */
sm_status signmuon_gated_mlp_backward(
    const void *dY, int64_t dy_stride, const void *X, int64_t x_stride,
    const void *Wg, const void *Wu, const void *Wd, const float *pre,
    int32_t dtype, int32_t act, int64_t rows, int64_t dim, int64_t hidden,
    void *dX, void *dWg, void *dWu, void *dWd, int32_t dw_dtype,
    int32_t accumulate, void *ws, size_t ws_bytes, hipStream_t stream);

/*
 * Softmax cross entropy of a linear output layer, whose logits Z = X W^T
 * (rows x vocab) are not kept: with t = targets[r],
 *   lse[r] = log(sum_v exp(Z[r,v])),  loss_r = lse[r] - Z[r,t] >= 0.
 * Row r of X starts at element r * x_stride (x_stride >= dim); W: contiguous
 * vocab x dim; both of `dtype`.  targets: rows integers of target_bits (32 or
 * 64) bits.  A row whose target is `ignore` (any integer) counts nowhere,
 * whatever it holds, and has loss_r = lse[r] = 0; a target that is neither
 * `ignore` nor in [0, vocab) makes its row's loss and gradients NaN.
 * loss: float32, loss_r of every row (SM_LOSS_ROWS), or one value: their sum
 * (SM_LOSS_SUM) or their mean over the rows that are not ignored
 * (SM_LOSS_MEAN; 0 where none is left).  lse: float32[rows], for the backward
 * pass.  0 <= rows <= 2^22, 1 <= dim <= 2^16, 1 <= vocab <= 2^20.
 * ws: signmuon_linear_cross_entropy_workspace() bytes (backward = 1 for the
 * backward call), 256-byte aligned; NULL where that is 0.  Its contents on
 * entry do not matter.  The query returns SIZE_MAX for arguments outside the
 * limits.
 */
enum { SM_LOSS_ROWS = 0, SM_LOSS_SUM = 1, SM_LOSS_MEAN = 2 };
size_t signmuon_linear_cross_entropy_workspace(int64_t rows, int64_t dim,
                                               int64_t vocab, int32_t dtype,
                                               int32_t backward);
sm_status signmuon_linear_cross_entropy(
    const void *X, int64_t x_stride, const void *W, int32_t dtype,
    const void *targets, int32_t target_bits, int64_t rows, int64_t dim,
    int64_t vocab, int64_t ignore, int32_t reduction, float *loss, float *lse,
    void *ws, size_t ws_bytes, hipStream_t stream);

/*
 * Its backward pass for the gradient dloss of loss (float32 on the device:
 * [rows] for SM_LOSS_ROWS, else one value): with
 *   G[r,v] = (exp(Z[r,v] - lse[r]) - [v = t]) * dloss (/ rows that count),
 *   dX = G W,  dW = G^T X.
 * The logits are computed again, a piece of the vocabulary after the other; a
 * piece of G is held in the workspace, rounded to `dtype`; in bfloat16, where
 * rows are at most 128 or rows times dim at most 2^16, to a sum of two values.
 * A factor that all rows share multiplies the results instead.  lse is what the
 * forward pass wrote.  dX: contiguous rows x dim of `dtype`, zeros in ignored
 * rows; it may be X itself if X is contiguous.  dW: contiguous vocab x dim of
 * dw_dtype; accumulate = 1 adds to what is there (float32 only).  Either may
 * be NULL: it is not computed then.
 */
sm_status signmuon_linear_cross_entropy_backward(
    const float *dloss, const void *X, int64_t x_stride, const void *W,
    int32_t dtype, const void *targets, int32_t target_bits, const float *lse,
    int64_t rows, int64_t dim, int64_t vocab, int64_t ignore,
    int32_t reduction, void *dX, void *dW, int32_t dw_dtype,
    int32_t accumulate, void *ws, size_t ws_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* SIGNMUON_LAYERS_H */
