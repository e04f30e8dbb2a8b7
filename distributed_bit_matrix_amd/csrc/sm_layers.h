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

}  // namespace sm
