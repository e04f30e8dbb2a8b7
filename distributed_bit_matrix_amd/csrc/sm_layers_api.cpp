// C ABI of the layer operators (signmuon_layers.h): argument validation.
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "sm_layers.h"

using namespace sm;

namespace {

constexpr int64_t kMaxDim = 1 << 20;                 // cols, dim, vocab
constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxTokens = (int64_t)1 << 30;
constexpr int64_t kMaxSorted = (int64_t)1 << 27;     // 256 runs of 2^19, 2^15 tokens a wave
constexpr int64_t kMaxMmRows = (int64_t)1 << 22;     // rows, widths of the matrix products
constexpr int64_t kMaxMmDim = 1 << 16;
constexpr int64_t kMaxCodesCols = 16384;              // rows that the norm holds in registers
constexpr int64_t kMaxStride = (int64_t)1 << 39;      // elements; past any memory

bool dtype_ok(int32_t d) { return d == SM_F32 || d == SM_BF16; }
bool aligned(const void* p, int32_t dtype) {
  return (uintptr_t)p % (dtype == SM_F32 ? 4 : 2) == 0;
}
bool in(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v <= hi; }
// a row stride that memory can hold, and whose last row has a 63-bit byte offset
bool stride_ok(int64_t stride, int64_t rows, int64_t cols) {
  return in(stride, cols, kMaxStride) && stride <= ((int64_t)1 << 60) / rows;
}
// whether none of `out` (null: not wanted) is one of `in`, or another of `out`
bool apart(std::initializer_list<const void*> out, std::initializer_list<const void*> in) {
  for (const void* const* o = out.begin(); o != out.end(); ++o) {
    if (!*o) continue;
    for (const void* i : in)
      if (*o == i) return false;
    for (const void* const* p = out.begin(); p != o; ++p)
      if (*o == *p) return false;
  }
  return true;
}
bool workspace_ok(const void* ws, size_t have, size_t need) {
  return need == 0 || (ws && have >= need && (uintptr_t)ws % 256 == 0);
}

}  // namespace

extern "C" {

sm_status signmuon_layer_norm(const void* X, int32_t x_dtype, int64_t x_stride,
                              const void* gamma, const void* beta, int32_t w_dtype,
                              int64_t rows, int64_t cols, float eps, void* Y, float* mean,
                              float* rstd, hipStream_t stream) {
  if (!dtype_ok(x_dtype) || !dtype_ok(w_dtype)) return SM_EINVAL;
  if (!in(rows, 0, kMaxRows) || !in(cols, 1, kMaxDim)) return SM_EINVAL;
  if (!std::isfinite(eps) || eps < 0.f) return SM_EINVAL;
  if (rows == 0) return SM_OK;
  if (!X || !Y || !stride_ok(x_stride, rows, cols)) return SM_EINVAL;
  if (X == Y && x_stride != cols) return SM_EINVAL;
  if (!aligned(X, x_dtype) || !aligned(Y, x_dtype) || !aligned(gamma, w_dtype) ||
      !aligned(beta, w_dtype) || !aligned(mean, SM_F32) || !aligned(rstd, SM_F32))
    return SM_EINVAL;
  const NormArgs a{X, x_stride, x_dtype, w_dtype, gamma, beta, rows, cols, eps, Y, mean, rstd};
  return launch_norm(a, stream) == hipSuccess ? SM_OK : SM_EHIP;
}

size_t signmuon_layer_norm_backward_workspace(int64_t rows, int64_t cols) {
  if (!in(rows, 0, kMaxRows) || !in(cols, 1, kMaxDim)) return SIZE_MAX;
  return norm_grad_workspace(rows, cols);
}

sm_status signmuon_layer_norm_backward(const void* dY, int64_t dy_stride, const void* X,
                                       int32_t x_dtype, int64_t x_stride, const void* gamma,
                                       int32_t w_dtype, const float* mean, const float* rstd,
                                       int64_t rows, int64_t cols, void* dX, void* dgamma,
                                       void* dbeta, int32_t dw_dtype, int32_t accumulate,
                                       void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!dtype_ok(x_dtype) || !dtype_ok(w_dtype) || !dtype_ok(dw_dtype)) return SM_EINVAL;
  if (!in(rows, 0, kMaxRows) || !in(cols, 1, kMaxDim)) return SM_EINVAL;
  if (!in(accumulate, 0, 1) || (accumulate && dw_dtype != SM_F32)) return SM_EINVAL;
  if (!dX && !dgamma && !dbeta) return SM_OK;
  if (rows > 0) {
    if (!dY || !X || !mean || !rstd) return SM_EINVAL;
    if (!stride_ok(dy_stride, rows, cols) || !stride_ok(x_stride, rows, cols)) return SM_EINVAL;
    if (dX && (dX == X || (dX == dY && dy_stride != cols))) return SM_EINVAL;
    if (!aligned(dY, x_dtype) || !aligned(X, x_dtype) || !aligned(gamma, w_dtype) ||
        !aligned(mean, SM_F32) || !aligned(rstd, SM_F32) || !aligned(dX, x_dtype))
      return SM_EINVAL;
  }
  if (!aligned(dgamma, dw_dtype) || !aligned(dbeta, dw_dtype)) return SM_EINVAL;
  if (!workspace_ok(ws, ws_bytes, norm_grad_workspace(rows, cols))) return SM_EWORKSPACE;
  if (dgamma && dgamma == dbeta) return SM_EINVAL;
  // (one launch for few rows reads gamma and the statistics and writes all results)
  if (rows > 0 && (!apart({dX, dgamma, dbeta}, {X, gamma, mean, rstd}) ||
                   !apart({dgamma, dbeta}, {dY})))
    return SM_EINVAL;
  const NormGradArgs a{dY, X, dy_stride, x_stride, x_dtype, w_dtype, dw_dtype, accumulate,
                       gamma, mean, rstd, rows, cols, dX, dgamma, dbeta, ws};
  return launch_norm_grad(a, stream) == hipSuccess ? SM_OK : SM_EHIP;
}

sm_status signmuon_embedding(const void* W, int32_t w_dtype, int64_t vocab, int64_t dim,
                             const void* tokens, int32_t token_bits, int64_t n, float scale,
                             void* Y, int32_t y_dtype, hipStream_t stream) {
  if (!dtype_ok(w_dtype) || !dtype_ok(y_dtype)) return SM_EINVAL;
  if (token_bits != 32 && token_bits != 64) return SM_EINVAL;
  if (!in(n, 0, kMaxTokens) || !in(vocab, 1, kMaxDim) || !in(dim, 1, kMaxDim)) return SM_EINVAL;
  if (!std::isfinite(scale)) return SM_EINVAL;
  if (n == 0) return SM_OK;
  if (!W || !tokens || !Y) return SM_EINVAL;
  if (!aligned(W, w_dtype) || !aligned(Y, y_dtype) || (uintptr_t)tokens % (token_bits / 8))
    return SM_EINVAL;
  const EmbedArgs a{W, w_dtype, y_dtype, token_bits, vocab, dim, n, tokens, scale, Y};
  return launch_embed(a, stream) == hipSuccess ? SM_OK : SM_EHIP;
}

size_t signmuon_embedding_backward_workspace(int64_t n, int64_t vocab, int64_t dim) {
  if (!in(n, 0, kMaxSorted) || !in(vocab, 1, kMaxDim) || !in(dim, 1, kMaxDim)) return SIZE_MAX;
  return embed_grad_workspace(n, vocab, dim);
}

sm_status signmuon_embedding_backward(const void* dY, int32_t dy_dtype, int64_t dy_stride,
                                      const void* tokens, int32_t token_bits, int64_t n,
                                      int64_t padding, float scale, void* dW, int32_t dw_dtype,
                                      int64_t vocab, int64_t dim, int32_t accumulate, void* ws,
                                      size_t ws_bytes, hipStream_t stream) {
  if (!dtype_ok(dy_dtype) || !dtype_ok(dw_dtype)) return SM_EINVAL;
  if (token_bits != 32 && token_bits != 64) return SM_EINVAL;
  if (!in(n, 0, kMaxSorted) || !in(vocab, 1, kMaxDim) || !in(dim, 1, kMaxDim)) return SM_EINVAL;
  if (!in(padding, -1, vocab - 1) || !std::isfinite(scale)) return SM_EINVAL;
  if (!in(accumulate, 0, 1) || (accumulate && dw_dtype != SM_F32)) return SM_EINVAL;
  if (n == 0 && accumulate) return SM_OK;
  if (!dW || !aligned(dW, dw_dtype)) return SM_EINVAL;
  if (n > 0) {
    if (!dY || !tokens || !stride_ok(dy_stride, n, dim)) return SM_EINVAL;
    if (!aligned(dY, dy_dtype) || (uintptr_t)tokens % (token_bits / 8)) return SM_EINVAL;
  }
  if (!workspace_ok(ws, ws_bytes, embed_grad_workspace(n, vocab, dim))) return SM_EWORKSPACE;
  const EmbedGradArgs a{dY, dy_dtype, dw_dtype, token_bits, accumulate, dy_stride, tokens, n,
                        padding, scale, dW, vocab, dim, ws};
  return launch_embed_grad(a, stream) == hipSuccess ? SM_OK : SM_EHIP;
}

static sm_status rms_call(const void* X, int64_t x_stride, const void* R, int64_t r_stride,
                          int32_t x_dtype, const void* gamma, int32_t w_dtype, int64_t rows,
                          int64_t cols, float eps, int64_t block, void* H, void* Y, bool codes,
                          float* scales, float* rstd, hipStream_t stream) {
  if (!dtype_ok(x_dtype) || !dtype_ok(w_dtype)) return SM_EINVAL;
  if (!in(rows, 0, kMaxRows) || !in(cols, 1, codes ? kMaxCodesCols : kMaxDim)) return SM_EINVAL;
  if (!std::isfinite(eps) || eps < 0.f) return SM_EINVAL;
  if (codes && block != 0 && block != 128) return SM_EINVAL;
  if (rows == 0) return SM_OK;
  if (!X || !Y || !stride_ok(x_stride, rows, cols)) return SM_EINVAL;
  if (R && (!H || !stride_ok(r_stride, rows, cols))) return SM_EINVAL;
  if (codes && (!scales || Y == X)) return SM_EINVAL;
  if (Y == X && x_stride != cols) return SM_EINVAL;
  if (R && ((H == X && x_stride != cols) || (H == R && r_stride != cols))) return SM_EINVAL;
  const void* sum = R ? H : nullptr;
  if (!apart({Y, sum, rstd, codes ? scales : nullptr}, {gamma}) ||
      !apart({rstd, codes ? scales : nullptr}, {X, R}) || (R && Y == R))
    return SM_EINVAL;
  if (!aligned(X, x_dtype) || !aligned(R, x_dtype) || !aligned(gamma, w_dtype) ||
      !aligned(rstd, SM_F32) || !aligned(scales, SM_F32) || (R && !aligned(H, x_dtype)) ||
      (!codes && !aligned(Y, x_dtype)))
    return SM_EINVAL;
  const RmsArgs a{X, R, x_stride, r_stride, x_dtype, w_dtype, gamma, rows, cols, eps,
                  (int32_t)block, H, Y, scales, rstd};
  return launch_rms(a, stream) == hipSuccess ? SM_OK : SM_EHIP;
}

sm_status signmuon_rms_norm(const void* X, int64_t x_stride, const void* R, int64_t r_stride,
                            int32_t x_dtype, const void* gamma, int32_t w_dtype, int64_t rows,
                            int64_t cols, float eps, void* H, void* Y, float* rstd,
                            hipStream_t stream) {
  return rms_call(X, x_stride, R, r_stride, x_dtype, gamma, w_dtype, rows, cols, eps, 0, H, Y,
                  false, nullptr, rstd, stream);
}

sm_status signmuon_rms_norm_e4m3(const void* X, int64_t x_stride, const void* R, int64_t r_stride,
                                 int32_t x_dtype, const void* gamma, int32_t w_dtype, int64_t rows,
                                 int64_t cols, float eps, int64_t block, void* H, void* Q,
                                 float* scales, float* rstd, hipStream_t stream) {
  return rms_call(X, x_stride, R, r_stride, x_dtype, gamma, w_dtype, rows, cols, eps, block, H, Q,
                  true, scales, rstd, stream);
}

size_t signmuon_rms_norm_backward_workspace(int64_t rows, int64_t cols) {
  if (!in(rows, 0, kMaxRows) || !in(cols, 1, kMaxDim)) return SIZE_MAX;
  return rms_grad_workspace(rows, cols);
}

sm_status signmuon_rms_norm_backward(const void* dY, int64_t dy_stride, const void* H,
                                     int64_t h_stride, const void* dH, int64_t dh_stride,
                                     int32_t x_dtype, const void* gamma, int32_t w_dtype,
                                     const float* rstd, int64_t rows, int64_t cols, void* dX,
                                     void* dgamma, int32_t dw_dtype, int32_t accumulate, void* ws,
                                     size_t ws_bytes, hipStream_t stream) {
  if (!dtype_ok(x_dtype) || !dtype_ok(w_dtype) || !dtype_ok(dw_dtype)) return SM_EINVAL;
  if (!in(rows, 0, kMaxRows) || !in(cols, 1, kMaxDim)) return SM_EINVAL;
  if (!in(accumulate, 0, 1) || (accumulate && dw_dtype != SM_F32)) return SM_EINVAL;
  if (!dX && !dgamma) return SM_OK;
  if (rows > 0) {
    if (!dY || !H || !rstd) return SM_EINVAL;
    if (!stride_ok(dy_stride, rows, cols) || !stride_ok(h_stride, rows, cols)) return SM_EINVAL;
    if (dH && !stride_ok(dh_stride, rows, cols)) return SM_EINVAL;
    if (dX && ((dX == dY && dy_stride != cols) || (dX == dH && dh_stride != cols)))
      return SM_EINVAL;
    // (one launch for few rows reads gamma and writes dgamma)
    if (!apart({dX, dgamma}, {H, gamma, rstd}) || !apart({dgamma}, {dY, dH})) return SM_EINVAL;
    if (!aligned(dY, x_dtype) || !aligned(H, x_dtype) || !aligned(dH, x_dtype) ||
        !aligned(gamma, w_dtype) || !aligned(rstd, SM_F32) || !aligned(dX, x_dtype))
      return SM_EINVAL;
  }
  if (!aligned(dgamma, dw_dtype)) return SM_EINVAL;
  if (!workspace_ok(ws, ws_bytes, rms_grad_workspace(rows, cols))) return SM_EWORKSPACE;
  const RmsGradArgs a{dY, H, dH, dy_stride, h_stride, dh_stride, x_dtype, w_dtype, dw_dtype,
                      accumulate, gamma, rstd, rows, cols, dX, dgamma, ws};
  return launch_rms_grad(a, stream) == hipSuccess ? SM_OK : SM_EHIP;
}

size_t signmuon_gated_mlp_workspace(int64_t rows, int64_t dim, int64_t hidden, int32_t dtype,
                                    int32_t backward) {
  if (!dtype_ok(dtype) || !in(backward, 0, 1) || !in(rows, 0, kMaxMmRows) ||
      !in(dim, 1, kMaxMmDim) || !in(hidden, 1, kMaxMmDim))
    return SIZE_MAX;
  return ffn_workspace(rows, dim, hidden, dtype, backward);
}

sm_status signmuon_gated_mlp(const void* X, int64_t x_stride, const void* Wg, const void* Wu,
                             const void* Wd, int32_t dtype, int32_t act, int64_t rows, int64_t dim,
                             int64_t hidden, void* Y, float* pre, void* ws, size_t ws_bytes,
                             hipStream_t stream) {
  if (!dtype_ok(dtype) || !in(act, SM_ACT_SILU, SM_ACT_GELU)) return SM_EINVAL;
  if (!in(rows, 0, kMaxMmRows) || !in(dim, 1, kMaxMmDim) || !in(hidden, 1, kMaxMmDim))
    return SM_EINVAL;
  if (rows == 0) return SM_OK;
  if (!X || !Wg || !Wu || !Wd || !Y || !stride_ok(x_stride, rows, dim)) return SM_EINVAL;
  for (const void* in : {X, Wg, Wu, Wd})
    if (Y == in || pre == in) return SM_EINVAL;
  if (pre == Y) return SM_EINVAL;
  if (!aligned(X, dtype) || !aligned(Wg, dtype) || !aligned(Wu, dtype) || !aligned(Wd, dtype) ||
      !aligned(Y, dtype) || !aligned(pre, SM_F32))
    return SM_EINVAL;
  if (!workspace_ok(ws, ws_bytes, ffn_workspace(rows, dim, hidden, dtype, false)))
    return SM_EWORKSPACE;
  const FfnArgs a{X, x_stride, Wg, Wu, Wd, dtype, act, rows, dim, hidden, Y, pre, ws};
  return launch_ffn(a, stream) == hipSuccess ? SM_OK : SM_EHIP;
}

sm_status signmuon_gated_mlp_backward(const void* dY, int64_t dy_stride, const void* X,
                                      int64_t x_stride, const void* Wg, const void* Wu,
                                      const void* Wd, const float* pre, int32_t dtype, int32_t act,
                                      int64_t rows, int64_t dim, int64_t hidden, void* dX,
                                      void* dWg, void* dWu, void* dWd, int32_t dw_dtype,
                                      int32_t accumulate, void* ws, size_t ws_bytes,
                                      hipStream_t stream) {
  if (!dtype_ok(dtype) || !dtype_ok(dw_dtype) || !in(act, SM_ACT_SILU, SM_ACT_GELU))
    return SM_EINVAL;
  if (!in(rows, 0, kMaxMmRows) || !in(dim, 1, kMaxMmDim) || !in(hidden, 1, kMaxMmDim))
    return SM_EINVAL;
  if (!in(accumulate, 0, 1) || (accumulate && dw_dtype != SM_F32)) return SM_EINVAL;
  if (!dX && !dWg && !dWu && !dWd) return SM_OK;
  if (rows > 0) {
    if (!dY || !X || !Wg || !Wu || !Wd || !pre) return SM_EINVAL;
    if (!stride_ok(dy_stride, rows, dim) || !stride_ok(x_stride, rows, dim)) return SM_EINVAL;
    for (const void* in : {dY, X, Wg, Wu, Wd, (const void*)pre})
      for (const void* out : {dX, dWg, dWu, dWd})
        if (out && out == in) return SM_EINVAL;
    if (!aligned(dY, dtype) || !aligned(X, dtype) || !aligned(Wg, dtype) || !aligned(Wu, dtype) ||
        !aligned(Wd, dtype) || !aligned(pre, SM_F32) || !aligned(dX, dtype))
      return SM_EINVAL;
  }
  if (!aligned(dWg, dw_dtype) || !aligned(dWu, dw_dtype) || !aligned(dWd, dw_dtype))
    return SM_EINVAL;
  const void* out[] = {dX, dWg, dWu, dWd};
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < i; ++j)
      if (out[i] && out[i] == out[j]) return SM_EINVAL;
  if (!workspace_ok(ws, ws_bytes, ffn_workspace(rows, dim, hidden, dtype, true)))
    return SM_EWORKSPACE;
  const FfnGradArgs a{dY, dy_stride, X, x_stride, Wg, Wu, Wd, pre, dtype, act, rows, dim, hidden,
                      dX, dWg, dWu, dWd, dw_dtype, accumulate, ws};
  return launch_ffn_grad(a, stream) == hipSuccess ? SM_OK : SM_EHIP;
}

size_t signmuon_linear_cross_entropy_workspace(int64_t rows, int64_t dim, int64_t vocab,
                                               int32_t dtype, int32_t backward) {
  if (!dtype_ok(dtype) || !in(backward, 0, 1) || !in(rows, 0, kMaxMmRows) ||
      !in(dim, 1, kMaxMmDim) || !in(vocab, 1, kMaxDim))
    return SIZE_MAX;
  return loss_workspace(rows, dim, vocab, dtype, backward);
}

sm_status signmuon_linear_cross_entropy(const void* X, int64_t x_stride, const void* W,
                                        int32_t dtype, const void* targets, int32_t target_bits,
                                        int64_t rows, int64_t dim, int64_t vocab, int64_t ignore,
                                        int32_t reduction, float* loss, float* lse, void* ws,
                                        size_t ws_bytes, hipStream_t stream) {
  if (!dtype_ok(dtype) || !in(reduction, SM_LOSS_ROWS, SM_LOSS_MEAN)) return SM_EINVAL;
  if (target_bits != 32 && target_bits != 64) return SM_EINVAL;
  if (!in(rows, 0, kMaxMmRows) || !in(dim, 1, kMaxMmDim) || !in(vocab, 1, kMaxDim))
    return SM_EINVAL;
  if (rows == 0 && reduction == SM_LOSS_ROWS) return SM_OK;
  if (!loss || !aligned(loss, SM_F32)) return SM_EINVAL;
  if (rows > 0) {
    if (!X || !W || !targets || !lse || !stride_ok(x_stride, rows, dim)) return SM_EINVAL;
    if (loss == lse) return SM_EINVAL;
    for (const void* out : {loss, lse})
      if (out == X || out == W || out == targets) return SM_EINVAL;
    if (!aligned(X, dtype) || !aligned(W, dtype) || !aligned(lse, SM_F32) ||
        (uintptr_t)targets % (target_bits / 8))
      return SM_EINVAL;
  }
  if (!workspace_ok(ws, ws_bytes, loss_workspace(rows, dim, vocab, dtype, false)))
    return SM_EWORKSPACE;
  const LossArgs a{X, x_stride, W, dtype, targets, target_bits, rows, dim, vocab, ignore,
                   reduction, loss, lse, ws};
  return launch_loss(a, stream) == hipSuccess ? SM_OK : SM_EHIP;
}

sm_status signmuon_linear_cross_entropy_backward(
    const float* dloss, const void* X, int64_t x_stride, const void* W, int32_t dtype,
    const void* targets, int32_t target_bits, const float* lse, int64_t rows, int64_t dim,
    int64_t vocab, int64_t ignore, int32_t reduction, void* dX, void* dW, int32_t dw_dtype,
    int32_t accumulate, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!dtype_ok(dtype) || !dtype_ok(dw_dtype) || !in(reduction, SM_LOSS_ROWS, SM_LOSS_MEAN))
    return SM_EINVAL;
  if (target_bits != 32 && target_bits != 64) return SM_EINVAL;
  if (!in(rows, 0, kMaxMmRows) || !in(dim, 1, kMaxMmDim) || !in(vocab, 1, kMaxDim))
    return SM_EINVAL;
  if (!in(accumulate, 0, 1) || (accumulate && dw_dtype != SM_F32)) return SM_EINVAL;
  if (!dX && !dW) return SM_OK;
  if (rows > 0) {
    if (!dloss || !X || !W || !targets || !lse || !stride_ok(x_stride, rows, dim))
      return SM_EINVAL;
    if (dX == X && x_stride != dim) return SM_EINVAL;
    if (!apart({dX, dW}, {W, targets, lse, dloss}) || !apart({dW}, {X})) return SM_EINVAL;
    if (!aligned(dloss, SM_F32) || !aligned(X, dtype) || !aligned(W, dtype) ||
        !aligned(lse, SM_F32) || !aligned(dX, dtype) || (uintptr_t)targets % (target_bits / 8))
      return SM_EINVAL;
  }
  if (!aligned(dW, dw_dtype) || (dX && dX == dW)) return SM_EINVAL;
  if (!workspace_ok(ws, ws_bytes, loss_workspace(rows, dim, vocab, dtype, true)))
    return SM_EWORKSPACE;
  const LossGradArgs a{dloss, X, x_stride, W, dtype, targets, target_bits, lse, rows, dim,
                       vocab, ignore, reduction, dX, dW, dw_dtype, accumulate, ws};
  return launch_loss_grad(a, stream) == hipSuccess ? SM_OK : SM_EHIP;
}

}  // extern "C"
