// Launchers of the layer operators (signmuon_layers.h), with checked
// arguments.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "signmuon_layers.h"

namespace sm {

struct NormArgs {
  const void* X;
  int64_t x_stride;
  int32_t x_dtype, w_dtype;
  const void *gamma, *beta;
  int64_t rows, cols;
  float eps;
  void* Y;
  float *mean, *rstd;
};
hipError_t launch_norm(const NormArgs& a, hipStream_t s);   // rows > 0

struct NormGradArgs {
  const void *dY, *X;
  int64_t dy_stride, x_stride;
  int32_t x_dtype, w_dtype, dw_dtype, accumulate;
  const void* gamma;
  const float *mean, *rstd;
  int64_t rows, cols;
  void *dX, *dgamma, *dbeta;
  void* ws;
};
size_t norm_grad_workspace(int64_t rows, int64_t cols);
hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t s);

struct EmbedArgs {
  const void* W;
  int32_t w_dtype, y_dtype, token_bits;
  int64_t vocab, dim, n;
  const void* tokens;
  float scale;
  void* Y;
};
hipError_t launch_embed(const EmbedArgs& a, hipStream_t s);   // n > 0

struct EmbedGradArgs {
  const void* dY;
  int32_t dy_dtype, dw_dtype, token_bits, accumulate;
  int64_t dy_stride;
  const void* tokens;
  int64_t n, padding;
  float scale;
  void* dW;
  int64_t vocab, dim;
  void* ws;
};
size_t embed_grad_workspace(int64_t n, int64_t vocab, int64_t dim);
hipError_t launch_embed_grad(const EmbedGradArgs& a, hipStream_t s);

struct RmsArgs {
  const void *X, *R;       // R: the residual stream, or null
  int64_t x_stride, r_stride;
  int32_t x_dtype, w_dtype;
  const void* gamma;
  int64_t rows, cols;
  float eps;
  int32_t block;           // columns of a scale: 128, or 0 for a whole row
  void *H, *Y;             // Y: of X's type, or codes where scales is not null
  float *scales, *rstd;
};
hipError_t launch_rms(const RmsArgs& a, hipStream_t s);   // rows > 0

struct RmsGradArgs {
  const void *dY, *H, *dH;
  int64_t dy_stride, h_stride, dh_stride;
  int32_t x_dtype, w_dtype, dw_dtype, accumulate;
  const void* gamma;
  const float* rstd;
  int64_t rows, cols;
  void *dX, *dgamma;
  void* ws;
};
size_t rms_grad_workspace(int64_t rows, int64_t cols);
hipError_t launch_rms_grad(const RmsGradArgs& a, hipStream_t s);

struct LossArgs {
  const void* X;
  int64_t x_stride;
  const void* W;
  int32_t dtype;
  const void* targets;
  int32_t target_bits;
  int64_t rows, dim, vocab, ignore;
  int32_t reduction;
  float *loss, *lse;
  void* ws;
};
size_t loss_workspace(int64_t rows, int64_t dim, int64_t vocab, int32_t dtype, bool backward);
hipError_t launch_loss(const LossArgs& a, hipStream_t s);   // rows > 0 for SM_LOSS_ROWS

struct LossGradArgs {
  const float* dloss;
  const void* X;
  int64_t x_stride;
  const void* W;
  int32_t dtype;
  const void* targets;
  int32_t target_bits;
  const float* lse;
  int64_t rows, dim, vocab, ignore;
  int32_t reduction;
  void *dX, *dW;
  int32_t dw_dtype, accumulate;
  void* ws;
};
hipError_t launch_loss_grad(const LossGradArgs& a, hipStream_t s);

struct FfnArgs {
  const void* X;
  int64_t x_stride;
  const void *Wg, *Wu, *Wd;
  int32_t dtype, act;
  int64_t rows, dim, hidden;
  void* Y;
  float* pre;
  void* ws;
};
size_t ffn_workspace(int64_t rows, int64_t dim, int64_t hidden, int32_t dtype, bool backward);
hipError_t launch_ffn(const FfnArgs& a, hipStream_t s);   // rows > 0

struct FfnGradArgs {
  const void* dY;
  int64_t dy_stride;
  const void* X;
  int64_t x_stride;
  const void *Wg, *Wu, *Wd;
  const float* pre;
  int32_t dtype, act;
  int64_t rows, dim, hidden;
  void *dX, *dWg, *dWu, *dWd;
  int32_t dw_dtype, accumulate;
  void* ws;
};
hipError_t launch_ffn_grad(const FfnGradArgs& a, hipStream_t s);

}  // namespace sm
