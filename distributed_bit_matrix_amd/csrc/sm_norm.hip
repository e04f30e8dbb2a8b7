// Layer norm of the rows of a matrix, forward and backward
// (signmuon_layers.h).  No floating-point atomics: every sum has an order
// that the sizes alone decide.
//
// Rows live in registers: a group of LANES threads holds one row as NV pieces
// of 16 bytes a thread, so a row is read from memory once, the squares are
// taken of deviations from the finished mean (a difference of squares would
// lose a large mean's variance), and the result is written from registers.
// Both passes are bound by HBM.
#include <algorithm>

#include "sm_layers.h"
#include "sm_rows.h"

namespace sm {

// Sums of K values each over groups of LANES threads, in a fixed order; valid
// in every thread of the group.  Groups wider than a wave meet in LDS, where
// `turn` alternates between two buffers: one barrier a sum is enough, since a
// buffer is written again only after the barrier of the sum in between.
template <int LANES, int K>
__device__ __forceinline__ void group_sums(float (&v)[K], int& turn) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = lanes_sum<(LANES < 64 ? LANES : 64)>(v[k]);
  if constexpr (LANES > 64) {
    constexpr int W = LANES / 64, G = 512 / LANES > 0 ? 512 / LANES : 1;
    __shared__ float sh[2][G][K][W];
    const int g = threadIdx.x / LANES, w = threadIdx.x % LANES >> 6;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) sh[turn][g][k][w] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float t = sh[turn][g][k][0];
#pragma unroll
      for (int j = 1; j < W; ++j) t += sh[turn][g][k][j];
      v[k] = t;
    }
    turn ^= 1;
  }
}

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------
template <typename T, typename TW, int V, int LANES, int NV>
__global__ __launch_bounds__(LANES > 256 ? LANES : 256) void k_norm(
    const T* X, int64_t xs, const TW* gamma, const TW* beta, int64_t rows, int cols, float eps,
    T* Y, float* mean, float* rstd) {
  constexpr int GROUPS = LANES > 256 ? 1 : 256 / LANES;
  const int lane = threadIdx.x % LANES;
  const Place<V> last(((NV - 1) * LANES + lane) * V, cols);   // only the last piece can be cut
  const float inv = 1.0f / cols;
  int turn = 0;
  for (int64_t r = (int64_t)blockIdx.x * GROUPS + threadIdx.x / LANES; r < rows;
       r += (int64_t)gridDim.x * GROUPS) {
    Piece<T, V> in[NV];
    Piece<TW, V> g[NV], b[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j)
      in[j].load(X + r * xs + (j < NV - 1 ? (j * LANES + lane) * V : last.c));
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = j < NV - 1 ? (j * LANES + lane) * V : last.c;
      if (gamma) g[j].load(gamma + c);
      if (beta) b[j].load(beta + c);
    }
    float x[NV][V];
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < V; ++k) {
        x[j][k] = in[j][k];
        s[0] += j < NV - 1 || k >= last.skip ? x[j][k] : 0.f;
      }
    group_sums<LANES, 1>(s, turn);
    const float mu = s[0] / cols;
    s[0] = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < V; ++k) {
        x[j][k] = j < NV - 1 || k >= last.skip ? x[j][k] - mu : 0.f;
        s[0] += x[j][k] * x[j][k];
      }
    group_sums<LANES, 1>(s, turn);
    const float rs = 1.0f / sqrtf(s[0] * inv + eps);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int k = 0; k < V; ++k)
        x[j][k] = x[j][k] * rs * (gamma ? g[j][k] : 1.f) + (beta ? b[j][k] : 0.f);
      if (j < NV - 1) store_vec<V>(Y + r * cols + (j * LANES + lane) * V, x[j]);
      else store_own<V>(Y + r * cols + last.c, last.skip, x[j]);
    }
    if (lane == 0) {
      if (mean) mean[r] = mu;
      if (rstd) rstd[r] = rs;
    }
  }
}

// Sum over a block of 1024 threads in a fixed order; valid in every thread.
__device__ __forceinline__ float block_total(float v) {
  __shared__ float sh[16];
  v = lanes_sum<64>(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  float t = 0.f;
#pragma unroll
  for (int k = 0; k < 16; ++k) t += sh[k];
  return t;
}

// Rows too long for registers: one block per row, which is read once for the
// mean, once for the squared deviations from it and once for the result.
template <typename T, typename TW>
__global__ __launch_bounds__(1024) void k_norm_long(const T* X, int64_t xs, const TW* gamma,
                                                    const TW* beta, int64_t rows, int cols,
                                                    float eps, T* Y, float* mean, float* rstd) {
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const T* x = X + r * xs;
    T* y = Y + r * cols;
    float s = 0.f;
    for (int c = threadIdx.x; c < cols; c += 1024) s += to_f32(x[c]);
    const float mu = block_total(s) / cols;
    float q = 0.f;
    for (int c = threadIdx.x; c < cols; c += 1024) {
      const float d = to_f32(x[c]) - mu;
      q += d * d;
    }
    const float rs = 1.0f / sqrtf(block_total(q) / cols + eps);
    for (int c = threadIdx.x; c < cols; c += 1024)
      put(y + c, (to_f32(x[c]) - mu) * rs * (gamma ? to_f32(gamma[c]) : 1.f) +
                     (beta ? to_f32(beta[c]) : 0.f));
    if (threadIdx.x == 0) {
      if (mean) mean[r] = mu;
      if (rstd) rstd[r] = rs;
    }
  }
}

// ---------------------------------------------------------------------------
// Backward.  One pass over dY and X: a block takes every gridDim-th set of
// rows, writes their dX, and adds dY * xhat and dY of its columns up in
// registers; its groups' sums meet in LDS at the end, and k_norm_join adds the
// blocks' (part[block][2][cols]).
// ---------------------------------------------------------------------------
template <typename T, typename TW, int V, int LANES, int NV>
__global__ __launch_bounds__(LANES > 512 ? LANES : 512, 4) void k_norm_grad(
    const T* dY, int64_t dys, const T* X, int64_t xs, const TW* gamma, const float* mean,
    const float* rstd, int64_t rows, int cols, T* dX, float* part) {
  constexpr int THREADS = LANES > 512 ? LANES : 512, GROUPS = THREADS / LANES;
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const Place<V> last(((NV - 1) * LANES + lane) * V, cols);   // only the last piece can be cut
  const float inv = 1.0f / cols;
  int turn = 0;
  float w[NV][V], ag[NV][V], ab[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    Piece<TW, V> g;
    if (gamma) g.load(gamma + (j < NV - 1 ? (j * LANES + lane) * V : last.c));
#pragma unroll
    for (int k = 0; k < V; ++k) {
      w[j][k] = gamma ? g[k] : 1.f;
      ag[j][k] = ab[j][k] = 0.f;
    }
  }
  // where groups meet in barriers, all of a block's go through the same turns
  for (int64_t r0 = (int64_t)blockIdx.x * GROUPS; r0 < rows; r0 += (int64_t)gridDim.x * GROUPS) {
    const int64_t r = r0 + group;
    const bool live = r < rows;
    float s[2] = {0.f, 0.f};
    float g[NV][V], xh[NV][V];
    float rs = 0.f;
    if (live) {
      Piece<T, V> pd[NV], px[NV];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = j < NV - 1 ? (j * LANES + lane) * V : last.c;
        pd[j].load(dY + r * dys + c);
        px[j].load(X + r * xs + c);
      }
      const float mu = mean[r];
      rs = rstd[r];
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < V; ++k) {
          // what is not the lane's own counts as dY = 0, X = mean
          const bool own = j < NV - 1 || k >= last.skip;
          const float dy = own ? pd[j][k] : 0.f;
          xh[j][k] = own ? (px[j][k] - mu) * rs : 0.f;
          ag[j][k] += dy * xh[j][k];
          ab[j][k] += dy;
          g[j][k] = dy * w[j][k];
          s[0] += g[j][k];
          s[1] += g[j][k] * xh[j][k];
        }
    }
    if (!dX) continue;
    group_sums<LANES, 2>(s, turn);
    if (!live) continue;
    const float c1 = s[0] * inv, c2 = s[1] * inv;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int k = 0; k < V; ++k) g[j][k] = rs * (g[j][k] - c1 - xh[j][k] * c2);
      if (j < NV - 1) store_vec<V>(dX + r * cols + (j * LANES + lane) * V, g[j]);
      else store_own<V>(dX + r * cols + last.c, last.skip, g[j]);
    }
  }
  if (!part) return;
  float* out = part + (int64_t)blockIdx.x * 2 * cols;
  if constexpr (GROUPS == 1) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = j < NV - 1 ? (j * LANES + lane) * V : last.c;
      const int skip = j < NV - 1 ? 0 : last.skip;
      store_own<V>(out + c, skip, ag[j]);
      store_own<V>(out + cols + c, skip, ab[j]);
    }
  } else {
    // one column after the other of a piece, so that neighbouring lanes write
    // neighbouring words
    constexpr int SPAN = LANES * NV * V;
    __shared__ float sh[GROUPS * SPAN];
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < V; ++k)
          sh[group * SPAN + (j * V + k) * LANES + lane] = pass ? ab[j][k] : ag[j][k];
      __syncthreads();
      for (int q = threadIdx.x; q < SPAN; q += THREADS) {
        const int l = q % LANES, jk = q / LANES, j = jk / V, k = jk % V;
        const Place<V> at((j * LANES + l) * V, cols);
        if (k < at.skip) continue;
        float t = sh[q];
#pragma unroll 8
        for (int g = 1; g < GROUPS; ++g) t += sh[g * SPAN + q];
        out[pass * cols + at.c + k] = t;
      }
    }
  }
}

// dX of rows too long for registers.
template <typename T, typename TW>
__global__ __launch_bounds__(1024) void k_norm_grad_long(
    const T* dY, int64_t dys, const T* X, int64_t xs, const TW* gamma, const float* mean,
    const float* rstd, int64_t rows, int cols, T* dX) {
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const T* x = X + r * xs;
    const T* dy = dY + r * dys;
    T* dx = dX + r * cols;
    const float mu = mean[r], rs = rstd[r];
    float s1 = 0.f, s2 = 0.f;
    for (int c = threadIdx.x; c < cols; c += 1024) {
      const float g = to_f32(dy[c]) * (gamma ? to_f32(gamma[c]) : 1.f);
      s1 += g;
      s2 += g * ((to_f32(x[c]) - mu) * rs);
    }
    const float c1 = block_total(s1) / cols, c2 = block_total(s2) / cols;
    for (int c = threadIdx.x; c < cols; c += 1024) {
      const float g = to_f32(dy[c]) * (gamma ? to_f32(gamma[c]) : 1.f);
      const float xh = (to_f32(x[c]) - mu) * rs;
      put(dx + c, rs * (g - c1 - xh * c2));
    }
  }
}

// Column sums of dY * xhat and of dY over one run of such rows: 64 columns by
// 4 row lanes a block, to part[run][2][cols].
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

// dgamma (blockIdx.y = 0) and dbeta (1) from the blocks' sums: 32 columns by
// 32 lanes over the blocks.
template <typename TO>
__global__ __launch_bounds__(1024) void k_norm_join(const float* part, int blocks, int cols,
                                                    TO* dgamma, TO* dbeta, int accumulate) {
  __shared__ float sh[32][33];
  TO* out = blockIdx.y ? dbeta : dgamma;
  if (!out) return;
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + x;
  const float* p = part + (int64_t)blockIdx.y * cols + c;
  float s = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int b = y; b < blocks; b += 32) s += p[(int64_t)b * 2 * cols];
  }
  sh[y][x] = s;
  __syncthreads();
  if (y == 0 && c < cols) {
    for (int k = 1; k < 32; ++k) s += sh[k][x];
    put(out + c, accumulate ? to_f32(out[c]) + s : s);
  }
}

namespace {

constexpr int64_t kMaxBlocks = 1 << 16;   // larger grids loop
constexpr int kGradBlocks = 512;          // two blocks of 512 threads a CU

// Threads a row: the fewest that hold it in at most `most` pieces each.  0: too long.
// Rows shorter than a piece go entry by entry (8 threads).
int lanes_for(int64_t cols, int vec, int most) {
  for (int lanes : {8, 16, 32})
    if (cols <= lanes * vec) return lanes;
  for (int lanes : {64, 256, 1024})
    if (cols <= (int64_t)lanes * vec * most) return lanes;
  return 0;
}
int vec_of(int32_t dtype) { return dtype == SM_BF16 ? 8 : 4; }
// The backward pass holds five values an entry: 16 entries a thread.
int grad_lanes(int64_t cols, int32_t dtype) {
  return lanes_for(cols, vec_of(dtype), 16 / vec_of(dtype));
}

// Blocks whose partial sums k_norm_join adds.
int64_t grad_blocks(int64_t rows, int64_t cols, int32_t dtype) {
  const int lanes = grad_lanes(cols, dtype);
  if (lanes == 0) return std::min<int64_t>((rows + 63) / 64, 64);
  const int groups = lanes > 512 ? 1 : 512 / lanes;
  return std::min<int64_t>((rows + groups - 1) / groups, lanes > 512 ? 256 : kGradBlocks);
}

template <typename T, typename TW, int V, int LANES, int NV>
void norm_go(const NormArgs& a, hipStream_t s) {
  constexpr int THREADS = LANES > 256 ? LANES : 256, GROUPS = THREADS / LANES;
  const int64_t grid = std::min<int64_t>((a.rows + GROUPS - 1) / GROUPS, kMaxBlocks);
  hipLaunchKernelGGL((k_norm<T, TW, V, LANES, NV>), dim3((unsigned)grid), dim3(THREADS), 0, s,
                     (const T*)a.X, a.x_stride, (const TW*)a.gamma, (const TW*)a.beta, a.rows,
                     (int)a.cols, a.eps, (T*)a.Y, a.mean, a.rstd);
}

template <typename T, typename TW, int LANES>
void norm_pieces(const NormArgs& a, hipStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  const int64_t per = (int64_t)LANES * V;
  switch ((a.cols + per - 1) / per) {
    case 1: return norm_go<T, TW, V, LANES, 1>(a, s);
    case 2: return norm_go<T, TW, V, LANES, 2>(a, s);
    case 3: return norm_go<T, TW, V, LANES, 3>(a, s);
    default: return norm_go<T, TW, V, LANES, 4>(a, s);
  }
}

template <typename T, typename TW>
hipError_t norm(const NormArgs& a, hipStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  switch (lanes_for(a.cols, V, 4)) {
    case 8:
      if (a.cols < V) norm_go<T, TW, 1, 8, 1>(a, s);
      else norm_go<T, TW, V, 8, 1>(a, s);
      break;
    case 16: norm_go<T, TW, V, 16, 1>(a, s); break;
    case 32: norm_go<T, TW, V, 32, 1>(a, s); break;
    case 64: norm_pieces<T, TW, 64>(a, s); break;
    case 256: norm_pieces<T, TW, 256>(a, s); break;
    case 1024: norm_pieces<T, TW, 1024>(a, s); break;
    default:
      hipLaunchKernelGGL((k_norm_long<T, TW>), dim3((unsigned)std::min(a.rows, kMaxBlocks)),
                         dim3(1024), 0, s, (const T*)a.X, a.x_stride, (const TW*)a.gamma,
                         (const TW*)a.beta, a.rows, (int)a.cols, a.eps, (T*)a.Y, a.mean, a.rstd);
  }
  return hipGetLastError();
}

template <typename T, typename TW, int V, int LANES, int NV>
void norm_grad_go(const NormGradArgs& a, int64_t grid, float* part, hipStream_t s) {
  hipLaunchKernelGGL((k_norm_grad<T, TW, V, LANES, NV>), dim3((unsigned)grid),
                     dim3(LANES > 512 ? LANES : 512), 0, s, (const T*)a.dY, a.dy_stride,
                     (const T*)a.X, a.x_stride, (const TW*)a.gamma, a.mean, a.rstd, a.rows,
                     (int)a.cols, (T*)a.dX, part);
}

template <typename T, typename TW, int LANES>
void norm_grad_pieces(const NormGradArgs& a, int64_t grid, float* part, hipStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  const int64_t per = (int64_t)LANES * V;
  const int64_t nv = (a.cols + per - 1) / per;
  if constexpr (V == 8) {
    if (nv == 1) norm_grad_go<T, TW, V, LANES, 1>(a, grid, part, s);
    else norm_grad_go<T, TW, V, LANES, 2>(a, grid, part, s);
  } else {
    switch (nv) {
      case 1: return norm_grad_go<T, TW, V, LANES, 1>(a, grid, part, s);
      case 2: return norm_grad_go<T, TW, V, LANES, 2>(a, grid, part, s);
      case 3: return norm_grad_go<T, TW, V, LANES, 3>(a, grid, part, s);
      default: return norm_grad_go<T, TW, V, LANES, 4>(a, grid, part, s);
    }
  }
}

template <typename T, typename TW>
hipError_t norm_grad(const NormGradArgs& a, hipStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  const bool sums = a.dgamma || a.dbeta;
  const int64_t blocks = grad_blocks(a.rows, a.cols, a.x_dtype);
  float* part = sums ? (float*)a.ws : nullptr;
  hipError_t e;
  if (a.rows > 0) {
    switch (grad_lanes(a.cols, a.x_dtype)) {
      case 8:
        if (a.cols < V) norm_grad_go<T, TW, 1, 8, 1>(a, blocks, part, s);
        else norm_grad_go<T, TW, V, 8, 1>(a, blocks, part, s);
        break;
      case 16: norm_grad_go<T, TW, V, 16, 1>(a, blocks, part, s); break;
      case 32: norm_grad_go<T, TW, V, 32, 1>(a, blocks, part, s); break;
      case 64: norm_grad_pieces<T, TW, 64>(a, blocks, part, s); break;
      case 256: norm_grad_pieces<T, TW, 256>(a, blocks, part, s); break;
      case 1024: norm_grad_pieces<T, TW, 1024>(a, blocks, part, s); break;
      default:
        // the column sums first: dX may be dY
        if (sums) {
          const int64_t run = (a.rows + blocks - 1) / blocks;
          hipLaunchKernelGGL((k_norm_cols<T>),
                             dim3((unsigned)((a.cols + 63) / 64), (unsigned)blocks), dim3(256),
                             0, s, (const T*)a.dY, a.dy_stride, (const T*)a.X, a.x_stride,
                             a.mean, a.rstd, a.rows, (int)a.cols, run, part);
          if ((e = hipGetLastError()) != hipSuccess) return e;
        }
        if (a.dX)
          hipLaunchKernelGGL((k_norm_grad_long<T, TW>),
                             dim3((unsigned)std::min(a.rows, kMaxBlocks)), dim3(1024), 0, s,
                             (const T*)a.dY, a.dy_stride, (const T*)a.X, a.x_stride,
                             (const TW*)a.gamma, a.mean, a.rstd, a.rows, (int)a.cols,
                             (T*)a.dX);
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (sums && !(a.rows == 0 && a.accumulate)) {
    const dim3 grid((unsigned)((a.cols + 31) / 32), 2);
    if (a.dw_dtype == SM_BF16)
      hipLaunchKernelGGL((k_norm_join<bf16_t>), grid, dim3(1024), 0, s, part, (int)blocks,
                         (int)a.cols, (bf16_t*)a.dgamma, (bf16_t*)a.dbeta, a.accumulate);
    else
      hipLaunchKernelGGL((k_norm_join<float>), grid, dim3(1024), 0, s, part, (int)blocks,
                         (int)a.cols, (float*)a.dgamma, (float*)a.dbeta, a.accumulate);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace

size_t norm_grad_workspace(int64_t rows, int64_t cols) {
  const int64_t blocks = std::max(grad_blocks(rows, cols, SM_F32), grad_blocks(rows, cols, SM_BF16));
  return ((size_t)blocks * 2 * cols * 4 + 255) / 256 * 256;
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
