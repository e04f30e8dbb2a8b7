/*
 * signmuon_layers.h - C ABI of libsignmuon.so: the layers of a transformer
 * whose parameter gradients are not matrix products, forward and backward:
 * layer norm and embedding lookup, as HIP kernels for AMD Instinct MI355X
 * (gfx950).  Their weight gradients are sums over rows that end in the
 * float32 gradient G of signmuon_step; like every result of this library
 * they are bit-reproducible run to run, so that replicas which vote on one
 * bit per entry start from the same gradient.
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

#ifdef __cplusplus
}
#endif
#endif /* SIGNMUON_LAYERS_H */
