// C ABI of the layer operators (signmuon_layers.h): argument validation.
#include <cmath>
#include <cstdint>

#include "sm_layers.h"

using namespace sm;

namespace {

constexpr int64_t kMaxDim = 1 << 20;                 // cols, dim, vocab
constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxTokens = (int64_t)1 << 30;
constexpr int64_t kMaxSorted = (int64_t)1 << 27;     // 256 runs of 2^19, 2^15 tokens a wave
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

}  // extern "C"
