// Layer norm of the rows of a matrix, forward and backward
// (signmuon_layers.h).  No floating-point atomics: every sum has an order
// that the sizes alone decide.
#include "sm_layers.h"
#include "sm_rows.h"

namespace sm {

// Sum over a block of B threads in a fixed order; valid in every thread.
template <int B>
__device__ __forceinline__ float block_total(float v) {
  __shared__ float sh[B / 64];
  v = lanes_sum<64>(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  float t = 0.f;
#pragma unroll
  for (int k = 0; k < B / 64; ++k) t += sh[k];
  return t;
}

// One block per row, which is read once for the mean, once for the squared
// deviations from it and once for the result.
template <typename T, typename TW>
__global__ __launch_bounds__(256) void k_norm_loop(const T* X, int64_t xs, const TW* gamma,
                                                   const TW* beta, int64_t rows, int cols,
                                                   float eps, T* Y, float* mean, float* rstd) {
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const T* x = X + r * xs;
    T* y = Y + r * cols;
    float s = 0.f;
    for (int c = threadIdx.x; c < cols; c += 256) s += to_f32(x[c]);
    const float mu = block_total<256>(s) / cols;
    float q = 0.f;
    for (int c = threadIdx.x; c < cols; c += 256) {
      const float d = to_f32(x[c]) - mu;
      q += d * d;
    }
    const float rs = 1.0f / sqrtf(block_total<256>(q) / cols + eps);
    for (int c = threadIdx.x; c < cols; c += 256)
      put(y + c, (to_f32(x[c]) - mu) * rs * (gamma ? to_f32(gamma[c]) : 1.f) +
                     (beta ? to_f32(beta[c]) : 0.f));
    if (threadIdx.x == 0) {
      if (mean) mean[r] = mu;
      if (rstd) rstd[r] = rs;
    }
  }
}

template <typename T, typename TW>
__global__ __launch_bounds__(256) void k_norm_grad_loop(
    const T* dY, int64_t dys, const T* X, int64_t xs, const TW* gamma, const float* mean,
    const float* rstd, int64_t rows, int cols, T* dX) {
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const T* x = X + r * xs;
    const T* dy = dY + r * dys;
    T* dx = dX + r * cols;
    const float mu = mean[r], rs = rstd[r];
    float s1 = 0.f, s2 = 0.f;
    for (int c = threadIdx.x; c < cols; c += 256) {
      const float g = to_f32(dy[c]) * (gamma ? to_f32(gamma[c]) : 1.f);
      s1 += g;
      s2 += g * ((to_f32(x[c]) - mu) * rs);
    }
    const float c1 = block_total<256>(s1) / cols, c2 = block_total<256>(s2) / cols;
    for (int c = threadIdx.x; c < cols; c += 256) {
      const float g = to_f32(dy[c]) * (gamma ? to_f32(gamma[c]) : 1.f);
      const float xh = (to_f32(x[c]) - mu) * rs;
      put(dx + c, rs * (g - c1 - xh * c2));
    }
  }
}

// Column sums of dY * xhat and of dY over one run of rows: 64 columns by 4
// row lanes a block, partial sums to part[run][2][cols].
template <typename T>
__global__ __launch_bounds__(256) void k_norm_cols(const T* dY, int64_t dys, const T* X,
                                                   int64_t xs, const float* mean,
                                                   const float* rstd, int64_t rows, int cols,
                                                   int64_t run, float* part) {
  __shared__ float sh[2][4][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  const int64_t r0 = (int64_t)blockIdx.y * run;
  const int64_t r1 = r0 + run < rows ? r0 + run : rows;
  float sg = 0.f, sb = 0.f;
  if (c < cols)
    for (int64_t r = r0 + w; r < r1; r += 4) {
      const float dy = to_f32(dY[r * dys + c]);
      sg += dy * ((to_f32(X[r * xs + c]) - mean[r]) * rstd[r]);
      sb += dy;
    }
  sh[0][w][lane] = sg;
  sh[1][w][lane] = sb;
  __syncthreads();
  if (w < 2 && c < cols)
    part[((int64_t)blockIdx.y * 2 + w) * cols + c] =
        ((sh[w][0][lane] + sh[w][1][lane]) + sh[w][2][lane]) + sh[w][3][lane];
}

// dgamma and dbeta from the partial sums (or, with none, from nothing).
template <typename TO>
__global__ __launch_bounds__(256) void k_norm_join(const float* part, int runs, int cols,
                                                   TO* dgamma, TO* dbeta, int accumulate) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= cols) return;
  for (int k = 0; k < 2; ++k) {
    TO* out = k ? dbeta : dgamma;
    if (!out) continue;
    float s = 0.f;
    for (int b = 0; b < runs; ++b) s += part[((int64_t)b * 2 + k) * cols + c];
    put(out + c, accumulate ? to_f32(out[c]) + s : s);
  }
}

namespace {

constexpr int64_t kMaxBlocks = 1 << 16;   // larger grids loop

int64_t runs_of(int64_t rows) {
  int64_t n = (rows + 63) / 64;
  return n < 64 ? n : 64;
}

template <typename T, typename TW>
hipError_t norm(const NormArgs& a, hipStream_t s) {
  const int64_t grid = a.rows < kMaxBlocks ? a.rows : kMaxBlocks;
  hipLaunchKernelGGL((k_norm_loop<T, TW>), dim3((unsigned)grid), dim3(256), 0, s,
                     (const T*)a.X, a.x_stride, (const TW*)a.gamma, (const TW*)a.beta, a.rows,
                     (int)a.cols, a.eps, (T*)a.Y, a.mean, a.rstd);
  return hipGetLastError();
}

template <typename T, typename TW>
hipError_t norm_grad(const NormGradArgs& a, hipStream_t s) {
  hipError_t e;
  const int cols = (int)a.cols;
  // the column sums first: dX may be dY
  const bool sums = a.dgamma || a.dbeta;
  const int64_t runs = runs_of(a.rows);
  if (sums && runs > 0) {
    const int64_t run = (a.rows + runs - 1) / runs;
    hipLaunchKernelGGL((k_norm_cols<T>), dim3((cols + 63) / 64, (unsigned)runs), dim3(256), 0, s,
                       (const T*)a.dY, a.dy_stride, (const T*)a.X, a.x_stride, a.mean, a.rstd,
                       a.rows, cols, run, (float*)a.ws);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (sums && !(runs == 0 && a.accumulate)) {
    dim3 grid((cols + 255) / 256);
    if (a.dw_dtype == SM_BF16)
      hipLaunchKernelGGL((k_norm_join<bf16_t>), grid, dim3(256), 0, s, (const float*)a.ws,
                         (int)runs, cols, (bf16_t*)a.dgamma, (bf16_t*)a.dbeta, a.accumulate);
    else
      hipLaunchKernelGGL((k_norm_join<float>), grid, dim3(256), 0, s, (const float*)a.ws,
                         (int)runs, cols, (float*)a.dgamma, (float*)a.dbeta, a.accumulate);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (a.dX && a.rows > 0) {
    const int64_t grid = a.rows < kMaxBlocks ? a.rows : kMaxBlocks;
    hipLaunchKernelGGL((k_norm_grad_loop<T, TW>), dim3((unsigned)grid), dim3(256), 0, s,
                       (const T*)a.dY, a.dy_stride, (const T*)a.X, a.x_stride,
                       (const TW*)a.gamma, a.mean, a.rstd, a.rows, cols, (T*)a.dX);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace

size_t norm_grad_workspace(int64_t rows, int64_t cols) {
  return ((size_t)runs_of(rows) * 2 * cols * 4 + 255) / 256 * 256;
}

hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
  if (a.x_dtype == SM_BF16)
    return a.w_dtype == SM_BF16 ? norm<bf16_t, bf16_t>(a, s) : norm<bf16_t, float>(a, s);
  return a.w_dtype == SM_BF16 ? norm<float, bf16_t>(a, s) : norm<float, float>(a, s);
}

hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t s) {
  if (a.x_dtype == SM_BF16)
    return a.w_dtype == SM_BF16 ? norm_grad<bf16_t, bf16_t>(a, s)
                                : norm_grad<bf16_t, float>(a, s);
  return a.w_dtype == SM_BF16 ? norm_grad<float, bf16_t>(a, s) : norm_grad<float, float>(a, s);
}

}  // namespace sm
