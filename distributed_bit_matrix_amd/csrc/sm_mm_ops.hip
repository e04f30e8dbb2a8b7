// Operand copies of the matrix products and the join of split sums.
#include "sm_mm_ops.h"

namespace sm {

// A thread copies 8 entries of a row.  Bound by HBM.
template <typename T, int P>
__global__ __launch_bounds__(256) void k_planes(const T* src, int64_t stride, int64_t rows,
                                                int cols, int ld, const int32_t* list,
                                                const int32_t* count, bf16_t* dst) {
  const int64_t live = count ? *count : rows, plane = rows * ld;
  const int per = ld / 8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < live * per;
       i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / per;
    const int c = (int)(i - r * per) * 8;
    const T* p = src + (list ? (int64_t)list[r] : r) * stride + c;
    float v[8];
    if (c + 8 <= cols) {
      Piece<T, 8> in;
      in.load(p);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = in[k];
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = c + k < cols ? to_f32(p[k]) : 0.f;
    }
    float lo[4] = {v[0], v[1], v[2], v[3]}, hi[4] = {v[4], v[5], v[6], v[7]};
    store_planes<P>(dst + r * ld + c, plane, lo);
    store_planes<P>(dst + r * ld + c + 4, plane, hi);
  }
}

hipError_t launch_planes(const PlanesArgs& a, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  const int64_t work = a.rows * (a.ld / 8);
  const dim3 grid((unsigned)std::min<int64_t>((work + 255) / 256, 1 << 16));
  if (a.dtype == SM_BF16)
    hipLaunchKernelGGL((k_planes<bf16_t, 1>), grid, dim3(256), 0, s, (const bf16_t*)a.src,
                       a.stride, a.rows, a.cols, a.ld, a.list, a.count, a.dst);
  else
    hipLaunchKernelGGL((k_planes<float, 3>), grid, dim3(256), 0, s, (const float*)a.src, a.stride,
                       a.rows, a.cols, a.ld, a.list, a.count, a.dst);
  return hipGetLastError();
}

// A thread joins 4 entries of a row, in the order of the splits.
template <typename T>
__global__ __launch_bounds__(256) void k_join(JoinArgs a) {
  const int per = (a.cols + 3) / 4;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.rows * per;
       i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / per;
    const int c = (int)(i - r * per) * 4, here = a.cols - c;
    const int64_t at = a.pos ? a.pos[r] : r;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (at >= 0) {
      const float* p = a.part + at * a.part_ld + c;
      for (int k = 0; k < a.splits; ++k, p += a.split_step) {
        const f32x4_t t = *reinterpret_cast<const f32x4_t*>(p);
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] += t[q];
      }
    }
    T* o = static_cast<T*>(a.out) + r * a.ld + c;
    if (a.add) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (q < here) v[q] += to_f32(o[q]);
    }
    if (here >= 4) {
      store_vec<4>(o, v);
    } else {
      for (int q = 0; q < here; ++q) put(o + q, v[q]);
    }
  }
}

hipError_t launch_join(const JoinArgs& a, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  const int64_t work = a.rows * ((a.cols + 3) / 4);
  const dim3 grid((unsigned)std::min<int64_t>((work + 255) / 256, 1 << 16));
  if (a.dtype == SM_BF16) hipLaunchKernelGGL(k_join<bf16_t>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(k_join<float>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

template <typename T>
__global__ __launch_bounds__(256) void k_zero(T* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    p[i] = 0;
}

hipError_t launch_zero(void* p, int32_t dtype, int64_t n, hipStream_t s) {
  if (n == 0) return hipSuccess;
  const dim3 grid((unsigned)std::min<int64_t>((n + 255) / 256, 4096));
  if (dtype == SM_BF16) hipLaunchKernelGGL(k_zero<bf16_t>, grid, dim3(256), 0, s, (bf16_t*)p, n);
  else hipLaunchKernelGGL(k_zero<uint32_t>, grid, dim3(256), 0, s, (uint32_t*)p, n);
  return hipGetLastError();
}

}  // namespace sm
