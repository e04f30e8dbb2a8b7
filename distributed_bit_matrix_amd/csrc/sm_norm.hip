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
#include <type_traits>

#include "sm_layers.h"
#include "sm_norm_rows.h"

namespace sm {

// ---------------------------------------------------------------------------
// Forward.  16384 x 4096 float32 takes 80 to 90 us (6.0 to 6.7 TB/s), 12288 x
// 768 bfloat16 8.6 us (4.4 TB/s of what the cache holds: one load, two sums and
// one store deep, with nothing left to overlap).
// ---------------------------------------------------------------------------
template <typename T, typename TW, int V, int LANES, int NV, bool ONCE>
__global__ __launch_bounds__(LANES > 64 ? LANES : 256) void k_norm(
    const T* X, int64_t xs, const TW* gamma, const TW* beta, int64_t rows, int cols, float eps,
    T* Y, float* mean, float* rstd) {
  // groups wider than a wave are blocks of their own: they meet in barriers
  constexpr int GROUPS = LANES > 64 ? 1 : 256 / LANES;
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
      in[j].template load<ONCE>(X + r * xs + (j < NV - 1 ? (j * LANES + lane) * V : last.c));
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

// Count, mean and sum of squared deviations from it; joined with those of
// other values by the update that needs no difference of large squares
// (Chan, Golub and LeVeque 1979).  What joins nothing is taken as it is: its
// mean is no deviation, and the square of a large one is past float32.
struct Moments {
  float n, mu, m2;
  __device__ __forceinline__ void join(float nb, float mb, float qb) {
    const float t = n + nb, share = t > 0.f ? nb * __builtin_amdgcn_rcpf(t) : 0.f, d = mb - mu;
    mu = n > 0.f ? mu + d * share : mb;
    m2 = n > 0.f ? m2 + (qb + d * (d * (n * share))) : qb;
    n = t;
  }
};

// Rows too long for registers.  A block takes the moments of the whole row in
// one read, 32 entries a thread and step, and then writes its share of the row
// from a second read that comes from a cache.  gridDim.y blocks share a row
// where there are few: each takes the moments for itself, which costs no more
// time than one of them would (one CU's bandwidth), and no workspace.  Float32
// 2048 x 40000: 151 us (4.3 TB/s; 157 with 1024 threads, 173 with 256), 16 x
// 2^20: 66 us (65 and 98), one row of 2^20: 40 us (40 and 72).
constexpr int kLongThreads = 512;
template <typename T, typename TW, int V>
__global__ __launch_bounds__(kLongThreads) void k_norm_long(const T* X, int64_t xs, const TW* gamma,
                                                    const TW* beta, int64_t rows, int cols,
                                                    float eps, T* Y, float* mean, float* rstd) {
  constexpr int U = 32 / V, U2 = 16 / V, STEP = kLongThreads * V;
  __shared__ Moments sh[2][kLongThreads / 64];       // by turns, as in group_sums
  const int lane = threadIdx.x & 63;
  const int64_t pieces = (cols + V - 1) / V;
  const int p0 = (int)(pieces * blockIdx.y / gridDim.y);
  const int p1 = (int)(pieces * (blockIdx.y + 1) / gridDim.y);
  int turn = 0;
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const T* x = X + r * xs;
    T* y = Y + r * cols;
    Moments all = {0.f, 0.f, 0.f};
    for (int c = threadIdx.x * V; c < cols; c += U * STEP) {
      Piece<T, V> in[U];
#pragma unroll
      for (int u = 0; u < U; ++u) in[u].load(x + Place<V>(c + u * STEP, cols).c);
      float s = 0.f, q = 0.f;
      if (c + (U - 1) * STEP + V <= cols) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int k = 0; k < V; ++k) s += in[u][k];
        const float mb = s * (1.f / (U * V));
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int k = 0; k < V; ++k) q += (in[u][k] - mb) * (in[u][k] - mb);
        all.join(U * V, mb, q);
      } else {
        int own = 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int skip = Place<V>(c + u * STEP, cols).skip;
          own += V - skip;
#pragma unroll
          for (int k = 0; k < V; ++k) s += k >= skip ? in[u][k] : 0.f;
        }
        const float mb = s / own;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int skip = Place<V>(c + u * STEP, cols).skip;
#pragma unroll
          for (int k = 0; k < V; ++k) q += k >= skip ? (in[u][k] - mb) * (in[u][k] - mb) : 0.f;
        }
        all.join(own, mb, q);
      }
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1)
      all.join(__shfl_xor(all.n, o), __shfl_xor(all.mu, o), __shfl_xor(all.m2, o));
    if (lane == 0) sh[turn][threadIdx.x >> 6] = all;
    __syncthreads();
    all = sh[turn][0];
#pragma unroll
    for (int j = 1; j < kLongThreads / 64; ++j)
      all.join(sh[turn][j].n, sh[turn][j].mu, sh[turn][j].m2);
    turn ^= 1;
    const float mu = all.mu, rs = 1.0f / sqrtf(all.m2 / cols + eps);
    for (int p = p0 + threadIdx.x; p < p1; p += U2 * kLongThreads) {
      Piece<T, V> in[U2];
      Piece<TW, V> g[U2], b[U2];
#pragma unroll
      for (int u = 0; u < U2; ++u) {
        const int c = Place<V>((p + u * kLongThreads) * V, cols).c;
        in[u].load(x + c);
        if (gamma) g[u].load(gamma + c);
        if (beta) b[u].load(beta + c);
      }
#pragma unroll
      for (int u = 0; u < U2; ++u) {
        const Place<V> at((p + u * kLongThreads) * V, cols);
        float v[V];
#pragma unroll
        for (int k = 0; k < V; ++k)
          v[k] = (in[u][k] - mu) * rs * (gamma ? g[u][k] : 1.f) + (beta ? b[u][k] : 0.f);
        store_own<V>(y + at.c, p + u * kLongThreads < p1 ? at.skip : V, v);
      }
    }
    if (threadIdx.x == 0 && blockIdx.y == 0) {
      if (mean) mean[r] = mu;
      if (rstd) rstd[r] = rs;
    }
  }
}

// ---------------------------------------------------------------------------
// Backward.  One pass over dY and X: a block takes every gridDim-th set of
// rows, writes their dX, and adds dY * xhat and dY of its columns up in
// registers; its groups' sums meet in LDS at the end, and k_norm_join adds the
// blocks' (part[block][2][cols]).  16384 x 4096 bfloat16 takes 73 + 5 us (5.5
// TB/s), 12288 x 768 15 + 4 us: three rows a wave between the weights' load and
// the groups' join.  Fetching the next row ahead costs more (16.8 us).
// ---------------------------------------------------------------------------
// One row of the backward pass: g = dY gamma, xhat, and the lane's shares of
// the sums of g and g xhat; `each` sees every entry's dY and xhat.  Contraction
// is spelled out, so that the kernels that share this give dX the same bits.
template <int V, int LANES, int NV, bool ONCE, typename T, typename TW, typename F>
__device__ __forceinline__ void grad_row(const T* dY, const T* X, const Piece<TW, V> (&w)[NV],
                                         bool weighted, const Place<V>& last, float mu, float rs,
                                         float (&g)[NV][V], float (&xh)[NV][V], float (&s)[2],
                                         const F& each) {
#pragma clang fp contract(off)
  const int lane = threadIdx.x % LANES;
  Piece<T, V> pd[NV], px[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = j < NV - 1 ? (j * LANES + lane) * V : last.c;
    pd[j].template load<ONCE>(dY + c);
    px[j].template load<ONCE>(X + c);
  }
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int k = 0; k < V; ++k) {
      // what is not the lane's own counts as dY = 0, X = mean
      const bool own = j < NV - 1 || k >= last.skip;
      const float dy = own ? pd[j][k] : 0.f;
      xh[j][k] = own ? (px[j][k] - mu) * rs : 0.f;
      each(j, k, dy, xh[j][k]);
      g[j][k] = weighted ? dy * w[j][k] : dy;
      s[0] += g[j][k];
      s[1] = __builtin_fmaf(g[j][k], xh[j][k], s[1]);
    }
}
// dX = rstd (g - c1 - xhat c2)
template <int V, int LANES, int NV, typename T>
__device__ __forceinline__ void grad_store(T* dX, const Place<V>& last, float rs, float c1,
                                           float c2, float (&g)[NV][V],
                                           const float (&xh)[NV][V]) {
#pragma clang fp contract(off)
  const int lane = threadIdx.x % LANES;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int k = 0; k < V; ++k) g[j][k] = rs * __builtin_fmaf(-xh[j][k], c2, g[j][k] - c1);
    if (j < NV - 1) store_vec<V>(dX + (j * LANES + lane) * V, g[j]);
    else store_own<V>(dX + last.c, last.skip, g[j]);
  }
}

template <typename T, typename TW, int V, int LANES, int NV, bool ONCE>
__global__ __launch_bounds__(LANES > 512 ? LANES : 512, 4) void k_norm_grad(
    const T* dY, int64_t dys, const T* X, int64_t xs, const TW* gamma, const float* mean,
    const float* rstd, int64_t rows, int cols, T* dX, float* part) {
  constexpr int THREADS = LANES > 512 ? LANES : 512, GROUPS = THREADS / LANES;
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const Place<V> last(((NV - 1) * LANES + lane) * V, cols);   // only the last piece can be cut
  const float inv = 1.0f / cols;
  int turn = 0;
  Piece<TW, V> w[NV];
  float ag[NV][V], ab[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (gamma) w[j].load(gamma + (j < NV - 1 ? (j * LANES + lane) * V : last.c));
#pragma unroll
    for (int k = 0; k < V; ++k) ag[j][k] = ab[j][k] = 0.f;
  }
  // where groups meet in barriers, all of a block's go through the same turns
  for (int64_t r0 = (int64_t)blockIdx.x * GROUPS; r0 < rows; r0 += (int64_t)gridDim.x * GROUPS) {
    const int64_t r = r0 + group;
    const bool live = r < rows;
    float s[2] = {0.f, 0.f};
    float g[NV][V], xh[NV][V];
    float rs = 0.f;
    if (live) {
      rs = rstd[r];
      grad_row<V, LANES, NV, ONCE>(dY + r * dys, X + r * xs, w, gamma != nullptr, last, mean[r], rs,
                                   g, xh, s, [&](int j, int k, float dy, float x) {
                                     ag[j][k] = __builtin_fmaf(dy, x, ag[j][k]);
                                     ab[j][k] += dy;
                                   });
    }
    if (!dX) continue;
    group_sums<LANES, 2>(s, turn);
    if (live)
      grad_store<V, LANES, NV>(dX + r * cols, last, rs, s[0] * inv, s[1] * inv, g, xh);
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

// Rows too long for registers.  A first launch reads dY and X once: a wave
// takes kLongCols columns of a run of rows, keeps their column sums in
// registers (part[run][2][cols]) and leaves each row's shares of the sums of g
// and g xhat in share[row][wave].  A second one adds a row's shares, reads dY
// and X again and writes dX.  Bound by HBM: 2048 x 40000 in 312 us (float32,
// 5 passes over 328 MB at 5.3 TB/s) and 170 us (bfloat16).
constexpr int kLongCols = 512;

template <typename T, typename TW, int V>
__global__ __launch_bounds__(256) void k_norm_long_sums(
    const T* dY, int64_t dys, const T* X, int64_t xs, const TW* gamma, const float* mean,
    const float* rstd, int64_t rows, int cols, int64_t run, float* part, float2* share) {
  constexpr int NV = kLongCols / (64 * V), R = 4;      // R rows in flight
  const int lane = threadIdx.x & 63;
  const int waves = (cols + kLongCols - 1) / kLongCols;
  const int w = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  if (w >= waves) return;
  int c[NV], skip[NV];
  Piece<TW, V> wg[NV];
  float ag[NV][V], ab[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const Place<V> at(w * kLongCols + (j * 64 + lane) * V, cols);
    c[j] = at.c;
    skip[j] = at.skip;
    if (gamma) wg[j].load(gamma + at.c);
#pragma unroll
    for (int k = 0; k < V; ++k) ag[j][k] = ab[j][k] = 0.f;
  }
  const int64_t r0 = blockIdx.y * run, r1 = r0 + run < rows ? r0 + run : rows;
  for (int64_t r = r0; r < r1; r += R) {
    Piece<T, V> pd[R][NV], px[R][NV];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t at = r + i < r1 ? r + i : r;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        pd[i][j].load(dY + at * dys + c[j]);
        px[i][j].load(X + at * xs + c[j]);
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (r + i >= r1) break;
      const float mu = mean[r + i], rs = rstd[r + i];
      float s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const bool own = k >= skip[j];
          const float dy = own ? pd[i][j][k] : 0.f;
          const float xh = own ? (px[i][j][k] - mu) * rs : 0.f;
          ag[j][k] += dy * xh;
          ab[j][k] += dy;
          const float g = gamma ? dy * wg[j][k] : dy;
          s1 += g;
          s2 += g * xh;
        }
      if (share) {
        s1 = lanes_sum<64>(s1);
        s2 = lanes_sum<64>(s2);
        if (lane == 0) share[(r + i) * waves + w] = make_float2(s1, s2);
      }
    }
  }
  if (!part) return;
  float* out = part + (int64_t)blockIdx.y * 2 * cols;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    store_own<V>(out + c[j], skip[j], ag[j]);
    store_own<V>(out + cols + c[j], skip[j], ab[j]);
  }
}

template <typename T, typename TW, int V>
__global__ __launch_bounds__(256) void k_norm_grad_long(
    const T* dY, int64_t dys, const T* X, int64_t xs, const TW* gamma, const float* mean,
    const float* rstd, int64_t rows, int cols, const float2* share, T* dX) {
  constexpr int U = 16 / V;
  const int lane = threadIdx.x & 63;
  const int waves = (cols + kLongCols - 1) / kLongCols;
  const int c0 = (blockIdx.x * U * 256 + threadIdx.x) * V;
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
    Piece<T, V> pd[U], px[U];
    Piece<TW, V> wg[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = Place<V>(c0 + u * 256 * V, cols).c;
      pd[u].load(dY + r * dys + c);
      px[u].load(X + r * xs + c);
      if (gamma) wg[u].load(gamma + c);
    }
    float s1 = 0.f, s2 = 0.f;
#pragma unroll 4
    for (int k = lane; k < waves; k += 64) {
      const float2 v = share[r * waves + k];
      s1 += v.x;
      s2 += v.y;
    }
    const float c1 = lanes_sum<64>(s1) / cols, c2 = lanes_sum<64>(s2) / cols;
    const float mu = mean[r], rs = rstd[r];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Place<V> at(c0 + u * 256 * V, cols);
      float v[V];
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float g = gamma ? pd[u][k] * wg[u][k] : pd[u][k];
        v[k] = rs * (g - c1 - (px[u][k] - mu) * rs * c2);
      }
      store_own<V>(dX + r * cols + at.c, at.skip, v);
    }
  }
}

// Few rows, in one launch: the first row_blocks blocks write dX as k_norm_grad
// does, the others take 16 columns each, by 32 lanes over the rows, and write
// dgamma and dbeta.  dY and X are read twice, the second time from the cache.
// Bound by its launch: 333 x 1001 float32 takes 3.6 us.
// (Where dX is dY the two kinds of blocks go in two launches.)
template <typename T, typename TW, typename TO, int V, int LANES, int NV>
__global__ __launch_bounds__(LANES > 512 ? LANES : 512) void k_norm_grad_few(
    const T* dY, int64_t dys, const T* X, int64_t xs, const TW* gamma, const float* mean,
    const float* rstd, int rows, int cols, T* dX, int row_blocks, TO* dgamma, TO* dbeta,
    int accumulate) {
  constexpr int THREADS = LANES > 512 ? LANES : 512, GROUPS = THREADS / LANES;
  if ((int)blockIdx.x < row_blocks) {
    const int lane = threadIdx.x % LANES;
    const int r = blockIdx.x * GROUPS + threadIdx.x / LANES;
    const int at = r < rows ? r : rows - 1;     // groups meet in barriers
    const Place<V> last(((NV - 1) * LANES + lane) * V, cols);
    int turn = 0;
    Piece<TW, V> w[NV];
    if (gamma)
#pragma unroll
      for (int j = 0; j < NV; ++j)
        w[j].load(gamma + (j < NV - 1 ? (j * LANES + lane) * V : last.c));
    const float rs = rstd[at], inv = 1.0f / cols;
    float s[2] = {0.f, 0.f};
    float g[NV][V], xh[NV][V];
    grad_row<V, LANES, NV, false>(dY + at * dys, X + at * xs, w, gamma != nullptr, last, mean[at],
                                  rs, g, xh, s, [](int, int, float, float) {});
    group_sums<LANES, 2>(s, turn);
    if (r < rows)
      grad_store<V, LANES, NV>(dX + (int64_t)r * cols, last, rs, s[0] * inv, s[1] * inv, g, xh);
    return;
  }
  constexpr int ROWS = THREADS / 16;
  __shared__ float sh[2][ROWS][17];
  const int x = threadIdx.x & 15, y = threadIdx.x >> 4;
  const int c = (blockIdx.x - row_blocks) * 16 + x;
  float sg = 0.f, sb = 0.f;
  if (c < cols) {
#pragma unroll 4
    for (int r = y; r < rows; r += ROWS) {
      const float dy = to_f32(dY[r * dys + c]);
      sg += dy * ((to_f32(X[r * xs + c]) - mean[r]) * rstd[r]);
      sb += dy;
    }
  }
  sh[0][y][x] = sg;
  sh[1][y][x] = sb;
  __syncthreads();
  // 16 lanes a column and sum: a wave has 4 of the 32
  const int l = threadIdx.x & 15, q = threadIdx.x >> 4;
  const int d = (blockIdx.x - row_blocks) * 16 + (q & 15);
  if (q >= 32) return;
  TO* out = q < 16 ? dgamma : dbeta;
  float t = 0.f;
#pragma unroll
  for (int k = 0; k < ROWS; k += 16) t += sh[q >> 4][l + k][q & 15];
  t = lanes_sum<16>(t);
  if (l == 0 && d < cols && out) put(out + d, accumulate ? to_f32(out[d]) + t : t);
}

// dgamma (blockIdx.y = 0) and dbeta (1) from the blocks' sums: C columns by
// 1024 / C lanes over the blocks.  32 columns read whole lines; 16 make enough
// blocks of narrow rows (16384 x 4096: 5.0 against 7.0 us, 12288 x 768: 3.9
// either way).
template <typename TO, int C>
__global__ __launch_bounds__(1024) void k_norm_join(const float* part, int blocks, int cols,
                                                    TO* dgamma, TO* dbeta, int accumulate) {
  constexpr int L = 1024 / C;
  __shared__ float sh[L][C + 1];
  TO* out = blockIdx.y ? dbeta : dgamma;
  if (!out) return;
  const int x = threadIdx.x % C, y = threadIdx.x / C;
  const int c = blockIdx.x * C + x;
  const float* p = part + (int64_t)blockIdx.y * cols + c;
  float s = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int b = y; b < blocks; b += L) s += p[(int64_t)b * 2 * cols];
  }
  sh[y][x] = s;
  __syncthreads();
  // 16 lanes a column
  if (threadIdx.x < 16 * C) {
    const int l = threadIdx.x & 15, q = threadIdx.x >> 4, d = blockIdx.x * C + q;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < L; k += 16) s += sh[l + k][q];
    s = lanes_sum<16>(s);
    if (l == 0 && d < cols) put(out + d, accumulate ? to_f32(out[d]) + s : s);
  }
}

// The same for few blocks (of few long rows): a thread a column.  One row of
// 2^20: 23 us in all, 115 with 32 lanes a column.
template <typename TO>
__global__ __launch_bounds__(256) void k_norm_join_few(const float* part, int blocks, int cols,
                                                       TO* dgamma, TO* dbeta, int accumulate) {
  TO* out = blockIdx.y ? dbeta : dgamma;
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (!out || c >= cols) return;
  float s = 0.f;
#pragma unroll 4
  for (int b = 0; b < blocks; ++b) s += part[((int64_t)b * 2 + blockIdx.y) * cols + c];
  put(out + c, accumulate ? to_f32(out[c]) + s : s);
}

namespace {

// Blocks whose partial sums k_norm_join adds.
int64_t grad_blocks(int64_t rows, int64_t cols, int32_t dtype) {
  const int lanes = grad_lanes(cols, dtype);
  if (lanes == 0)     // runs of rows: 16 waves a CU, at least 8 rows a wave
    return std::min((rows + 7) / 8, std::max<int64_t>(1, 4096 * kLongCols / cols));
  const int groups = lanes > 512 ? 1 : 512 / lanes;
  return std::min<int64_t>((rows + groups - 1) / groups, lanes > 512 ? 256 : kGradBlocks);
}

// Workspace: the blocks' column sums, and for long rows the rows' shares.
size_t column_bytes(int64_t blocks, int64_t cols) {
  return ((size_t)blocks * 2 * cols * 4 + 255) / 256 * 256;
}

template <typename T, typename TW, int V, int LANES, int NV>
void norm_go(const NormArgs& a, hipStream_t s) {
  constexpr int THREADS = LANES > 64 ? LANES : 256, GROUPS = THREADS / LANES;
  const int64_t grid = std::min<int64_t>((a.rows + GROUPS - 1) / GROUPS, kMaxBlocks);
  const auto kernel = 2 * a.rows * a.cols * (int64_t)sizeof(T) > kCacheBytes
                          ? k_norm<T, TW, V, LANES, NV, true>
                          : k_norm<T, TW, V, LANES, NV, false>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(THREADS), 0, s, (const T*)a.X,
                     a.x_stride, (const TW*)a.gamma, (const TW*)a.beta, a.rows, (int)a.cols,
                     a.eps, (T*)a.Y, a.mean, a.rstd);
}

template <typename T, typename TW, int LANES>
void norm_pieces(const NormArgs& a, hipStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  const int64_t per = (int64_t)LANES * V;
  constexpr int LEAST = LANES == 32 ? 2 : LANES == 64 && V == 4 ? 1 : 3;
  constexpr int MOST = LANES == 1024 && V == 8 ? 3 : 4;
  with_pieces<LEAST, MOST>((a.cols + per - 1) / per, [&](auto nv) {
    norm_go<T, TW, V, LANES, decltype(nv)::value>(a, s);
  });
}

template <typename T, typename TW>
hipError_t norm(const NormArgs& a, hipStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  switch (norm_lanes(a.cols, a.x_dtype)) {
    case 8:
      if (a.cols < V) norm_go<T, TW, 1, 8, 1>(a, s);
      else norm_go<T, TW, V, 8, 1>(a, s);
      break;
    case 16: norm_go<T, TW, V, 16, 1>(a, s); break;
    case 32:
      if (a.cols <= 32 * V) norm_go<T, TW, V, 32, 1>(a, s);
      else if constexpr (V == 8) norm_pieces<T, TW, 32>(a, s);
      break;
    case 64: norm_pieces<T, TW, 64>(a, s); break;
    case 128: norm_pieces<T, TW, 128>(a, s); break;
    case 256: norm_pieces<T, TW, 256>(a, s); break;
    case 512: norm_pieces<T, TW, 512>(a, s); break;
    case 1024: norm_pieces<T, TW, 1024>(a, s); break;
    default: {
      // blocks that share a row; in place they would read what others wrote
      const int64_t share =
          a.X == a.Y ? 1 : std::max<int64_t>(1, std::min(256 / a.rows, a.cols / 8192));
      hipLaunchKernelGGL((k_norm_long<T, TW, V>),
                         dim3((unsigned)std::min(a.rows, kMaxBlocks), (unsigned)share),
                         dim3(kLongThreads), 0, s, (const T*)a.X, a.x_stride, (const TW*)a.gamma,
                         (const TW*)a.beta, a.rows, (int)a.cols, a.eps, (T*)a.Y, a.mean, a.rstd);
    }
  }
  return hipGetLastError();
}

template <typename T, typename TW, int V, int LANES, int NV>
void norm_grad_go(const NormGradArgs& a, int64_t grid, float* part, hipStream_t s) {
  const auto kernel = 3 * a.rows * a.cols * (int64_t)sizeof(T) > kCacheBytes
                          ? k_norm_grad<T, TW, V, LANES, NV, true>
                          : k_norm_grad<T, TW, V, LANES, NV, false>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(LANES > 512 ? LANES : 512), 0, s,
                     (const T*)a.dY, a.dy_stride, (const T*)a.X, a.x_stride, (const TW*)a.gamma,
                     a.mean, a.rstd, a.rows, (int)a.cols, (T*)a.dX, part);
}

template <typename T, typename TW, int LANES>
void norm_grad_pieces(const NormGradArgs& a, int64_t grid, float* part, hipStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  const int64_t per = (int64_t)LANES * V;
  with_pieces<GradPieces<V, LANES>::kLeast, GradPieces<V, LANES>::kMost>(
      (a.cols + per - 1) / per, [&](auto nv) {
        norm_grad_go<T, TW, V, LANES, decltype(nv)::value>(a, grid, part, s);
      });
}

template <typename T, typename TW, typename TO, int V, int LANES, int NV>
void norm_grad_few_go(const NormGradArgs& a, hipStream_t s) {
  constexpr int THREADS = LANES > 512 ? LANES : 512, GROUPS = THREADS / LANES;
  const int row_blocks = a.dX ? (int)((a.rows + GROUPS - 1) / GROUPS) : 0;
  const int col_blocks = a.dgamma || a.dbeta ? (int)((a.cols + 15) / 16) : 0;
  const auto go = [&](int rows, int cols) {
    if (rows + cols > 0)
      hipLaunchKernelGGL((k_norm_grad_few<T, TW, TO, V, LANES, NV>),
                         dim3((unsigned)(rows + cols)), dim3(THREADS), 0, s, (const T*)a.dY,
                         a.dy_stride, (const T*)a.X, a.x_stride, (const TW*)a.gamma, a.mean,
                         a.rstd, (int)a.rows, (int)a.cols, (T*)a.dX, rows, (TO*)a.dgamma,
                         (TO*)a.dbeta, a.accumulate);
  };
  if (a.dX == a.dY) {
    go(0, col_blocks);
    go(row_blocks, 0);
  } else {
    go(row_blocks, col_blocks);
  }
}

template <typename T, typename TW, typename TO, int LANES>
void norm_grad_few_pieces(const NormGradArgs& a, hipStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  const int64_t per = (int64_t)LANES * V;
  with_pieces<GradPieces<V, LANES>::kLeast, GradPieces<V, LANES>::kMost>(
      (a.cols + per - 1) / per, [&](auto nv) {
        norm_grad_few_go<T, TW, TO, V, LANES, decltype(nv)::value>(a, s);
      });
}

template <typename T, typename TW, typename TO>
hipError_t norm_grad_few(const NormGradArgs& a, hipStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  switch (grad_lanes(a.cols, a.x_dtype)) {
    case 8:
      if (a.cols < V) norm_grad_few_go<T, TW, TO, 1, 8, 1>(a, s);
      else norm_grad_few_go<T, TW, TO, V, 8, 1>(a, s);
      break;
    case 16: norm_grad_few_go<T, TW, TO, V, 16, 1>(a, s); break;
    case 32: norm_grad_few_go<T, TW, TO, V, 32, 1>(a, s); break;
    case 64: norm_grad_few_pieces<T, TW, TO, 64>(a, s); break;
    case 128:       // bfloat16 goes from 64 to 256
      if constexpr (V == 4) norm_grad_few_pieces<T, TW, TO, 128>(a, s);
      break;
    case 256: norm_grad_few_pieces<T, TW, TO, 256>(a, s); break;
    case 512: norm_grad_few_pieces<T, TW, TO, 512>(a, s); break;
    default: norm_grad_few_pieces<T, TW, TO, 1024>(a, s); break;
  }
  return hipGetLastError();
}

// Whether k_norm_grad_few serves these rows.  Kernels alone, against the two
// launches: 1500 x 57 5.3 against 5.4 + 2.5 us, 2048 x 768 10.7 (float32 13.4)
// against 5.9 + 3.3 (6.8 + 3.5), 2048 x 2000 14.7 (18.0) against 13.7 + 4.5
// (13.0 + 4.4); the launch that it saves is 4 us of host time.  So it is the
// faster one for eager calls, which the host bounds at these sizes; replayed from
// a graph, 2048 x 768 takes 1.5 us more than the two would (float32 3.1).  4000 x
// 57: 11 against 4.4 + 3.5, 512 x 16384 in a loop of calls 61 against 57.
bool few(int64_t rows, int64_t cols) {
  return rows > 0 && rows <= 2048 && rows * cols <= ((int64_t)1 << 22) && cols <= 16384;
}

template <typename TO>
hipError_t norm_join(const NormGradArgs& a, const float* part, int64_t blocks, hipStream_t s) {
  if (blocks <= 16) {
    hipLaunchKernelGGL((k_norm_join_few<TO>), dim3((unsigned)((a.cols + 255) / 256), 2), dim3(256),
                       0, s, part, (int)blocks, (int)a.cols, (TO*)a.dgamma, (TO*)a.dbeta,
                       a.accumulate);
    return hipGetLastError();
  }
  const bool wide = a.cols > 2048;
  const int c = wide ? 32 : 16;
  hipLaunchKernelGGL((wide ? k_norm_join<TO, 32> : k_norm_join<TO, 16>),
                     dim3((unsigned)((a.cols + c - 1) / c), 2), dim3(1024), 0, s, part,
                     (int)blocks, (int)a.cols, (TO*)a.dgamma, (TO*)a.dbeta, a.accumulate);
  return hipGetLastError();
}

template <typename T, typename TW>
hipError_t norm_grad(const NormGradArgs& a, hipStream_t s) {
  if (few(a.rows, a.cols))
    return a.dw_dtype == SM_BF16 ? norm_grad_few<T, TW, bf16_t>(a, s)
                                 : norm_grad_few<T, TW, float>(a, s);
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
      case 128:     // bfloat16 goes from 64 to 256
        if constexpr (V == 4) norm_grad_pieces<T, TW, 128>(a, blocks, part, s);
        break;
      case 256: norm_grad_pieces<T, TW, 256>(a, blocks, part, s); break;
      case 512: norm_grad_pieces<T, TW, 512>(a, blocks, part, s); break;
      case 1024: norm_grad_pieces<T, TW, 1024>(a, blocks, part, s); break;
      default:
        // all of dY is read before dX, which may be dY, is written
        const int64_t run = (a.rows + blocks - 1) / blocks;
        float2* share = a.dX ? (float2*)((char*)a.ws + column_bytes(blocks, a.cols)) : nullptr;
        hipLaunchKernelGGL((k_norm_long_sums<T, TW, V>),
                           dim3((unsigned)((a.cols + 4 * kLongCols - 1) / (4 * kLongCols)),
                                (unsigned)blocks),
                           dim3(256), 0, s, (const T*)a.dY, a.dy_stride, (const T*)a.X,
                           a.x_stride, (const TW*)a.gamma, a.mean, a.rstd, a.rows, (int)a.cols,
                           run, part, share);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        if (a.dX)
          hipLaunchKernelGGL((k_norm_grad_long<T, TW, V>),
                             dim3((unsigned)((a.cols + 4095) / 4096),
                                  (unsigned)std::min<int64_t>(a.rows, 65535)),
                             dim3(256), 0, s, (const T*)a.dY, a.dy_stride, (const T*)a.X,
                             a.x_stride, (const TW*)a.gamma, a.mean, a.rstd, a.rows, (int)a.cols,
                             share, (T*)a.dX);
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (sums && !(a.rows == 0 && a.accumulate)) {
    return a.dw_dtype == SM_BF16 ? norm_join<bf16_t>(a, part, blocks, s)
                                 : norm_join<float>(a, part, blocks, s);
  }
  return hipSuccess;
}

}  // namespace

size_t norm_grad_workspace(int64_t rows, int64_t cols) {
  if (few(rows, cols)) return 0;
  const int64_t blocks =
      std::max(grad_blocks(rows, cols, SM_F32), grad_blocks(rows, cols, SM_BF16));
  const int64_t waves = (cols + kLongCols - 1) / kLongCols;
  return column_bytes(blocks, cols) + (grad_lanes(cols, SM_F32) ? 0 : (size_t)(rows * waves) * 8);
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
