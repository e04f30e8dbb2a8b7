// Root-mean-square norm of a residual stream (signmuon_layers.h), forward and
// backward, with an 8-bit output too.  Rows live in registers as in the layer
// norm (sm_norm_rows.h), so each array is read or written once; every sum has an
// order that the sizes alone decide.  Both passes are bound by HBM: 16384 x 4096
// bfloat16 with a residual 94 us (537 MB, 5.7 TB/s), to 8 bits 84 (470 MB, 5.6 TB/s),
// its backward pass 96 (537 MB, 5.6 TB/s) and 5 for the blocks' sums; 12288 x 768 15 and
// 4, by a block's start and end; one row of 4096 3.
#include "sm_layers.h"
#include "sm_norm_rows.h"

namespace sm {

constexpr float kE4m3Max = 448.f;
constexpr float kLeastScale = 0x1p-126f;

template <int CTRL>
__device__ __forceinline__ float dpp_max(float v) {
  return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF,
                                                             false)));
}
// Maximum over aligned groups of W lanes, as lanes_sum; NaN counts as nothing.
template <int W>
__device__ __forceinline__ float lanes_max(float v) {
  if constexpr (W >= 2) v = dpp_max<0xB1>(v);
  if constexpr (W >= 4) v = dpp_max<0x4E>(v);
  if constexpr (W >= 8) v = dpp_max<0x141>(v);
  if constexpr (W >= 16) v = dpp_max<0x140>(v);
  if constexpr (W >= 32) v = fmaxf(v, __shfl_xor(v, 16));
  if constexpr (W >= 64) v = fmaxf(v, __shfl_xor(v, 32));
  return v;
}
// Maximum over groups of LANES threads that are blocks of their own past a wave.
template <int LANES>
__device__ __forceinline__ float group_max(float v) {
  v = lanes_max<(LANES < 64 ? LANES : 64)>(v);
  if constexpr (LANES > 64) {
    __shared__ float sh[LANES / 64];
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < LANES / 64; ++j) v = fmaxf(v, sh[j]);
  }
  return v;
}

typedef uint32_t u32x2_a1 __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32_a1 __attribute__((aligned(1)));
// Codes of V values, nearest even, the lane's own to p.
template <int V>
__device__ __forceinline__ void store_codes(uint8_t* p, int skip, const float (&v)[V]) {
  if constexpr (V == 1) {
    if (skip == 0) *p = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[0], 0.f, 0, false);
  } else {
    uint32_t w[V / 4];
#pragma unroll
    for (int q = 0; q < V / 4; ++q) {
      int t = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * q], v[4 * q + 1], 0, false);
      w[q] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * q + 2], v[4 * q + 3], t, true);
    }
    if (skip == 0) {
      if constexpr (V == 8) *reinterpret_cast<u32x2_a1*>(p) = u32x2_a1{w[0], w[1]};
      else *reinterpret_cast<u32_a1*>(p) = w[0];
    } else if (skip < V) {
#pragma unroll
      for (int k = 1; k < V; ++k)
        if (k >= skip) p[k] = (uint8_t)(w[k / 4] >> (8 * (k & 3)));
    }
  }
}

// x + r in float32, rounded to the stream's type
template <typename T>
__device__ __forceinline__ float add_rounded(float x, float r) {
  if constexpr (sizeof(T) == 4) return x + r;
  else return bf16_to_f32(f32_to_bf16(x + r));
}

template <typename P, typename T>
__device__ __forceinline__ void load_once(P& p, const T* from, bool once) {
  if (once) p.template load<true>(from);
  else p.load(from);
}

// ---------------------------------------------------------------------------
// Forward.
// ---------------------------------------------------------------------------
template <typename T, typename TW, int V, int LANES, int NV, bool CODES>
__global__ __launch_bounds__(LANES > 64 ? LANES : 256) void k_rms(RmsArgs a, bool once) {
  // groups wider than a wave are blocks of their own: they meet in barriers
  constexpr int GROUPS = LANES > 64 ? 1 : 256 / LANES;
  const int lane = threadIdx.x % LANES, cols = (int)a.cols;
  const Place<V> last(((NV - 1) * LANES + lane) * V, cols);   // only the last piece can be cut
  const T *X = (const T*)a.X, *R = (const T*)a.R;
  const TW* gamma = (const TW*)a.gamma;
  T* H = (T*)a.H;
  int turn = 0;
  for (int64_t r = (int64_t)blockIdx.x * GROUPS + threadIdx.x / LANES; r < a.rows;
       r += (int64_t)gridDim.x * GROUPS) {
    Piece<T, V> in[NV], add[NV];
    Piece<TW, V> g[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = j < NV - 1 ? (j * LANES + lane) * V : last.c;
      load_once(in[j], X + r * a.x_stride + c, once);
      if (R) load_once(add[j], R + r * a.r_stride + c, once);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (gamma) g[j].load(gamma + (j < NV - 1 ? (j * LANES + lane) * V : last.c));
    float x[NV][V];
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        x[j][k] = R ? add_rounded<T>(in[j][k], add[j][k]) : in[j][k];
        s[0] += j < NV - 1 || k >= last.skip ? x[j][k] * x[j][k] : 0.f;
      }
      if (R) {
        if (j < NV - 1) store_vec<V>(H + r * cols + (j * LANES + lane) * V, x[j]);
        else store_own<V>(H + r * cols + last.c, last.skip, x[j]);
      }
    }
    group_sums<LANES, 1>(s, turn);
    const float rs = 1.0f / sqrtf(s[0] / cols + a.eps);
    // For codes only rstd's power of two multiplies the row, which rounds nothing: h
    // gamma may be past float32's range, or below it, where Y is not.  What is left of
    // rstd is 1 to 2 (or 1, where rstd is 0 or not finite).
    float by_row = rs, left = 1.f;
    if constexpr (CODES) {
      if (rs > 0.f && rs < INFINITY) {
        const uint32_t b = __float_as_uint(rs);
        by_row = __uint_as_float(b & 0x7F800000u);
        left = __uint_as_float((b & 0x007FFFFFu) | 0x3F800000u);
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < V; ++k) {
        x[j][k] *= by_row;
        if (gamma) x[j][k] *= g[j][k];
      }
    if constexpr (!CODES) {
      T* Y = (T*)a.Y + r * cols;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (j < NV - 1) store_vec<V>(Y + (j * LANES + lane) * V, x[j]);
        else store_own<V>(Y + last.c, last.skip, x[j]);
      }
    } else {
      // A code is of Y / scale, where rstd cancels: 448 h gamma / max |h gamma|, divided
      // with a correction, has the division's rounding and that of h gamma, which is
      // exact of bfloat16; each rounding can move a value across the middle between two
      // codes (by way of Y there are five).  Where Y nears the ends of float32's range, or
      // the scale is the least, by way of Y.
      // A block of 128 columns is a piece of W lanes; shorter groups have one.
      constexpr int W = 128 / V < LANES ? 128 / V : LANES;
      uint8_t* Y = (uint8_t*)a.Y + r * cols;
      float most[NV];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        most[j] = 0.f;
#pragma unroll
        for (int k = 0; k < V; ++k)
          if (j < NV - 1 || k >= last.skip) most[j] = fmaxf(most[j], fabsf(x[j][k]));
      }
      const int blocks = a.block ? (cols + 127) / 128 : 1;
      if (a.block == 0) {
        float all = most[0];
#pragma unroll
        for (int j = 1; j < NV; ++j) all = fmaxf(all, most[j]);
        all = group_max<LANES>(all);
#pragma unroll
        for (int j = 0; j < NV; ++j) most[j] = all;
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (a.block) most[j] = lanes_max<W>(most[j]);
        const float scale = fmaxf(most[j] * left / kE4m3Max, kLeastScale);
        const bool direct = scale > kLeastScale && most[j] > 1e-30f && most[j] < 1e30f;
        const float first = direct ? kE4m3Max : left, by = direct ? most[j] : scale, inv = 1.f / by;
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float u = x[j][k] * first, q = u * inv;
          x[j][k] = direct ? __builtin_fmaf(__builtin_fmaf(-q, by, u), inv, q) : q;
        }
        const int at = (j * LANES + lane) * V;
        if (at < cols && (a.block ? at % 128 == 0 : at == 0))
          a.scales[r * blocks + (a.block ? at / 128 : 0)] = scale;
        if (j < NV - 1) store_codes<V>(Y + at, 0, x[j]);
        else store_codes<V>(Y + last.c, last.skip, x[j]);
      }
    }
    if (lane == 0 && a.rstd) a.rstd[r] = rs;
  }
}

// Rows too long for registers: a block reads a row twice, the second time from a
// cache.  gridDim.y blocks share a row where there are few; each sums the squares
// for itself and writes its share.  In place one block has the row: what a cut
// piece reads of its neighbour's entries, written or not, is not used.
constexpr int kRmsThreads = 512;
template <typename T, typename TW, int V>
__global__ __launch_bounds__(kRmsThreads) void k_rms_long(RmsArgs a) {
  constexpr int U = 16 / V, STEP = kRmsThreads * V;
  const int cols = (int)a.cols;
  const T *X = (const T*)a.X, *R = (const T*)a.R;
  const TW* gamma = (const TW*)a.gamma;
  const int64_t pieces = (cols + V - 1) / V;
  const int p0 = (int)(pieces * blockIdx.y / gridDim.y);
  const int p1 = (int)(pieces * (blockIdx.y + 1) / gridDim.y);
  int turn = 0;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T *x = X + r * a.x_stride, *add = R ? R + r * a.r_stride : nullptr;
    T *h = R ? (T*)a.H + r * cols : nullptr, *y = (T*)a.Y + r * cols;
    float s[1] = {0.f};
    for (int c = threadIdx.x * V; c < cols; c += U * STEP) {
      Piece<T, V> in[U], ad[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = Place<V>(c + u * STEP, cols).c;
        in[u].load(x + at);
        if (R) ad[u].load(add + at);
      }
      float part = 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int skip = Place<V>(c + u * STEP, cols).skip;
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float v = R ? add_rounded<T>(in[u][k], ad[u][k]) : in[u][k];
          part += k >= skip ? v * v : 0.f;
        }
      }
      s[0] += part;
    }
    group_sums<kRmsThreads, 1>(s, turn);
    const float rs = 1.0f / sqrtf(s[0] / cols + a.eps);
    for (int p = p0 + threadIdx.x; p < p1; p += U * kRmsThreads) {
      Piece<T, V> in[U], ad[U];
      Piece<TW, V> g[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = Place<V>((p + u * kRmsThreads) * V, cols).c;
        in[u].load(x + c);
        if (R) ad[u].load(add + c);
        if (gamma) g[u].load(gamma + c);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const Place<V> at((p + u * kRmsThreads) * V, cols);
        const int skip = p + u * kRmsThreads < p1 ? at.skip : V;
        float v[V];
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = R ? add_rounded<T>(in[u][k], ad[u][k]) : in[u][k];
        if (R) store_own<V>(h + at.c, skip, v);
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = v[k] * rs * (gamma ? g[u][k] : 1.f);
        store_own<V>(y + at.c, skip, v);
      }
    }
    if (threadIdx.x == 0 && blockIdx.y == 0 && a.rstd) a.rstd[r] = rs;
  }
}

// ---------------------------------------------------------------------------
// Backward: g = dY gamma, xhat = H rstd, dX = dH + rstd (g - xhat c2), c2 the mean
// of g xhat.  One pass over dY, H and dH: a block takes every gridDim-th set of
// rows and adds dY xhat of its columns up in registers; its groups' sums meet in
// LDS at the end, and k_rms_join adds the blocks' (part[block][cols]).
// ---------------------------------------------------------------------------
// One row: xhat, g and the lane's share of the sum of g xhat; `each` sees every
// entry's dY and xhat.  Contraction is spelled out, so that the kernels that share
// this give dX the same bits.
template <int V, int LANES, int NV, typename T, typename TW, typename F>
__device__ __forceinline__ void rms_row(const T* dY, const T* H, const T* dH, bool once,
                                        const Piece<TW, V> (&w)[NV], bool weighted,
                                        const Place<V>& last, float rs, Piece<T, V> (&pa)[NV],
                                        float (&g)[NV][V], float (&xh)[NV][V], float (&s)[1],
                                        const F& each) {
#pragma clang fp contract(off)
  const int lane = threadIdx.x % LANES;
  Piece<T, V> pd[NV], px[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = j < NV - 1 ? (j * LANES + lane) * V : last.c;
    load_once(pd[j], dY + c, once);
    load_once(px[j], H + c, once);
    if (dH) load_once(pa[j], dH + c, once);
  }
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const bool own = j < NV - 1 || k >= last.skip;
      const float dy = own ? pd[j][k] : 0.f;
      xh[j][k] = own ? px[j][k] * rs : 0.f;
      each(j, k, dy, xh[j][k]);
      g[j][k] = weighted ? dy * w[j][k] : dy;
      s[0] = __builtin_fmaf(g[j][k], xh[j][k], s[0]);
    }
}
template <int V, int LANES, int NV, typename T>
__device__ __forceinline__ void rms_store(T* dX, const Place<V>& last, float rs, float c2,
                                          bool added, const Piece<T, V> (&pa)[NV],
                                          float (&g)[NV][V], const float (&xh)[NV][V]) {
#pragma clang fp contract(off)
  const int lane = threadIdx.x % LANES;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const float t = __builtin_fmaf(-xh[j][k], c2, g[j][k]);
      g[j][k] = added ? __builtin_fmaf(rs, t, pa[j][k]) : rs * t;
    }
    if (j < NV - 1) store_vec<V>(dX + (j * LANES + lane) * V, g[j]);
    else store_own<V>(dX + last.c, last.skip, g[j]);
  }
}

template <typename T, typename TW, int V, int LANES, int NV>
__global__ __launch_bounds__(LANES > 512 ? LANES : 512, 4) void k_rms_grad(RmsGradArgs a, bool once,
                                                                        float* part) {
  constexpr int THREADS = LANES > 512 ? LANES : 512, GROUPS = THREADS / LANES;
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES, cols = (int)a.cols;
  const Place<V> last(((NV - 1) * LANES + lane) * V, cols);   // only the last piece can be cut
  const float inv = 1.0f / cols;
  const T *dY = (const T*)a.dY, *H = (const T*)a.H, *dH = (const T*)a.dH;
  const TW* gamma = (const TW*)a.gamma;
  T* dX = (T*)a.dX;
  int turn = 0;
  Piece<TW, V> w[NV];
  float ag[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (gamma) w[j].load(gamma + (j < NV - 1 ? (j * LANES + lane) * V : last.c));
#pragma unroll
    for (int k = 0; k < V; ++k) ag[j][k] = 0.f;
  }
  // where groups meet in barriers, all of a block's go through the same turns
  for (int64_t r0 = (int64_t)blockIdx.x * GROUPS; r0 < a.rows;
       r0 += (int64_t)gridDim.x * GROUPS) {
    const int64_t r = r0 + group;
    const bool live = r < a.rows;
    float s[1] = {0.f};
    float g[NV][V], xh[NV][V];
    Piece<T, V> pa[NV];
    float rs = 0.f;
    if (live) {
      rs = a.rstd[r];
      rms_row<V, LANES, NV>(dY + r * a.dy_stride, H + r * a.h_stride,
                            dH && dX ? dH + r * a.dh_stride : (const T*)nullptr, once, w,
                            gamma != nullptr, last, rs, pa, g, xh, s,
                            [&](int j, int k, float dy, float x) {
                              ag[j][k] = __builtin_fmaf(dy, x, ag[j][k]);
                            });
    }
    if (!dX) continue;
    group_sums<LANES, 1>(s, turn);
    if (live)
      rms_store<V, LANES, NV>(dX + r * cols, last, rs, s[0] * inv, dH != nullptr, pa, g, xh);
  }
  if (!part) return;
  float* out = part + (int64_t)blockIdx.x * cols;
  if constexpr (GROUPS == 1) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      store_own<V>(out + (j < NV - 1 ? (j * LANES + lane) * V : last.c),
                   j < NV - 1 ? 0 : last.skip, ag[j]);
  } else {
    // one column after the other of a piece, so that neighbouring lanes write
    // neighbouring words
    constexpr int SPAN = LANES * NV * V;
    __shared__ float sh[GROUPS * SPAN];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < V; ++k) sh[group * SPAN + (j * V + k) * LANES + lane] = ag[j][k];
    __syncthreads();
    for (int q = threadIdx.x; q < SPAN; q += THREADS) {
      const int l = q % LANES, jk = q / LANES, j = jk / V, k = jk % V;
      const Place<V> at((j * LANES + l) * V, cols);
      if (k < at.skip) continue;
      float t = sh[q];
#pragma unroll 8
      for (int o = 1; o < GROUPS; ++o) t += sh[o * SPAN + q];
      out[at.c + k] = t;
    }
  }
}

// Rows too long for registers.  A first launch reads dY and H once: a wave takes
// kRmsCols columns of a run of rows, keeps their column sums (part[run][cols]) and
// leaves each row's share of the sum of g xhat in share[row][wave].  A second one
// adds a row's shares and writes dX.
constexpr int kRmsCols = 512;

template <typename T, typename TW, int V>
__global__ __launch_bounds__(256) void k_rms_long_sums(RmsGradArgs a, int64_t run, float* part,
                                                       float* share) {
  constexpr int NV = kRmsCols / (64 * V), R = 4;      // R rows in flight
  const int lane = threadIdx.x & 63, cols = (int)a.cols;
  const int waves = (cols + kRmsCols - 1) / kRmsCols;
  const int w = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  if (w >= waves) return;
  const T *dY = (const T*)a.dY, *H = (const T*)a.H;
  const TW* gamma = (const TW*)a.gamma;
  int c[NV], skip[NV];
  Piece<TW, V> wg[NV];
  float ag[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const Place<V> at(w * kRmsCols + (j * 64 + lane) * V, cols);
    c[j] = at.c;
    skip[j] = at.skip;
    if (gamma) wg[j].load(gamma + at.c);
#pragma unroll
    for (int k = 0; k < V; ++k) ag[j][k] = 0.f;
  }
  const int64_t r0 = blockIdx.y * run, r1 = r0 + run < a.rows ? r0 + run : a.rows;
  for (int64_t r = r0; r < r1; r += R) {
    Piece<T, V> pd[R][NV], px[R][NV];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t at = r + i < r1 ? r + i : r;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        pd[i][j].load(dY + at * a.dy_stride + c[j]);
        px[i][j].load(H + at * a.h_stride + c[j]);
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (r + i >= r1) break;
      const float rs = a.rstd[r + i];
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const bool own = k >= skip[j];
          const float dy = own ? pd[i][j][k] : 0.f, xh = own ? px[i][j][k] * rs : 0.f;
          ag[j][k] += dy * xh;
          s += (gamma ? dy * wg[j][k] : dy) * xh;
        }
      if (share) {
        s = lanes_sum<64>(s);
        if (lane == 0) share[(r + i) * waves + w] = s;
      }
    }
  }
  if (!part) return;
#pragma unroll
  for (int j = 0; j < NV; ++j) store_own<V>(part + blockIdx.y * a.cols + c[j], skip[j], ag[j]);
}

template <typename T, typename TW, int V>
__global__ __launch_bounds__(256) void k_rms_grad_long(RmsGradArgs a, const float* share) {
  constexpr int U = 16 / V;
  const int lane = threadIdx.x & 63, cols = (int)a.cols;
  const int waves = (cols + kRmsCols - 1) / kRmsCols;
  const int c0 = (blockIdx.x * U * 256 + threadIdx.x) * V;
  const T *dY = (const T*)a.dY, *H = (const T*)a.H, *dH = (const T*)a.dH;
  const TW* gamma = (const TW*)a.gamma;
  for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
    Piece<T, V> pd[U], px[U], pa[U];
    Piece<TW, V> wg[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = Place<V>(c0 + u * 256 * V, cols).c;
      pd[u].load(dY + r * a.dy_stride + c);
      px[u].load(H + r * a.h_stride + c);
      if (dH) pa[u].load(dH + r * a.dh_stride + c);
      if (gamma) wg[u].load(gamma + c);
    }
    float s = 0.f;
#pragma unroll 4
    for (int k = lane; k < waves; k += 64) s += share[r * waves + k];
    const float c2 = lanes_sum<64>(s) / cols, rs = a.rstd[r];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Place<V> at(c0 + u * 256 * V, cols);
      float v[V];
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float g = gamma ? pd[u][k] * wg[u][k] : pd[u][k];
        v[k] = rs * (g - px[u][k] * rs * c2) + (dH ? pa[u][k] : 0.f);
      }
      store_own<V>((T*)a.dX + r * cols + at.c, at.skip, v);
    }
  }
}

// Few rows, in one launch: the first row_blocks blocks write dX as k_rms_grad does,
// the others take 16 columns each, by 32 lanes over the rows.  dY and H are read
// twice, the second time from the cache.  (Where dX is dY the two kinds of blocks
// go in two launches.)
template <typename T, typename TW, typename TO, int V, int LANES, int NV>
__global__ __launch_bounds__(LANES > 512 ? LANES : 512) void k_rms_grad_few(RmsGradArgs a,
                                                                           int row_blocks) {
  constexpr int THREADS = LANES > 512 ? LANES : 512, GROUPS = THREADS / LANES;
  const int rows = (int)a.rows, cols = (int)a.cols;
  const T *dY = (const T*)a.dY, *H = (const T*)a.H, *dH = (const T*)a.dH;
  const TW* gamma = (const TW*)a.gamma;
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
    const float rs = a.rstd[at], inv = 1.0f / cols;
    float s[1] = {0.f};
    float g[NV][V], xh[NV][V];
    Piece<T, V> pa[NV];
    rms_row<V, LANES, NV>(dY + at * a.dy_stride, H + at * a.h_stride,
                          dH ? dH + at * a.dh_stride : (const T*)nullptr, false, w,
                          gamma != nullptr, last, rs, pa, g, xh, s, [](int, int, float, float) {});
    group_sums<LANES, 1>(s, turn);
    if (r < rows)
      rms_store<V, LANES, NV>((T*)a.dX + (int64_t)r * cols, last, rs, s[0] * inv, dH != nullptr, pa,
                              g, xh);
    return;
  }
  constexpr int ROWS = THREADS / 16;
  __shared__ float sh[ROWS][17];
  const int x = threadIdx.x & 15, y = threadIdx.x >> 4;
  const int c = (blockIdx.x - row_blocks) * 16 + x;
  float t = 0.f;
  if (c < cols) {
#pragma unroll 4
    for (int r = y; r < rows; r += ROWS)
      t += to_f32(dY[r * a.dy_stride + c]) * (to_f32(H[r * a.h_stride + c]) * a.rstd[r]);
  }
  sh[y][x] = t;
  __syncthreads();
  // 16 lanes a column
  const int l = threadIdx.x & 15, q = threadIdx.x >> 4;
  const int d = (blockIdx.x - row_blocks) * 16 + q;
  if (q >= 16) return;
  TO* out = (TO*)a.dgamma;
  t = 0.f;
#pragma unroll
  for (int k = 0; k < ROWS; k += 16) t += sh[l + k][q];
  t = lanes_sum<16>(t);
  if (l == 0 && d < cols) put(out + d, a.accumulate ? to_f32(out[d]) + t : t);
}

// dgamma from the blocks' sums: 16 columns by 64 lanes over the blocks; where there
// are few blocks (of few long rows) a thread a column.
template <typename TO>
__global__ __launch_bounds__(1024) void k_rms_join(const float* part, int blocks, int cols,
                                                   TO* out, int accumulate) {
  __shared__ float sh[64][17];
  const int x = threadIdx.x & 15, y = threadIdx.x >> 4;
  const int c = blockIdx.x * 16 + x;
  float s = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int b = y; b < blocks; b += 64) s += part[(int64_t)b * cols + c];
  }
  sh[y][x] = s;
  __syncthreads();
  if (threadIdx.x < 256) {
    const int l = threadIdx.x & 15, q = threadIdx.x >> 4, d = blockIdx.x * 16 + q;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < 64; k += 16) s += sh[l + k][q];
    s = lanes_sum<16>(s);
    if (l == 0 && d < cols) put(out + d, accumulate ? to_f32(out[d]) + s : s);
  }
}
template <typename TO>
__global__ __launch_bounds__(256) void k_rms_join_few(const float* part, int blocks, int cols,
                                                      TO* out, int accumulate) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= cols) return;
  float s = 0.f;
#pragma unroll 4
  for (int b = 0; b < blocks; ++b) s += part[(int64_t)b * cols + c];
  put(out + c, accumulate ? to_f32(out[c]) + s : s);
}

namespace {

// Calls f(V, LANES, NV) as constants for rows of `cols` entries in `lanes` threads
// (norm_lanes, grad_lanes); false where the row is too long for registers.
template <int V, int LANES, int LEAST, int MOST, typename F>
void shape_pieces(int64_t cols, const F& f) {
  const int64_t per = (int64_t)LANES * V;
  with_pieces<LEAST, MOST>((cols + per - 1) / per, [&](auto nv) {
    f(std::integral_constant<int, V>(), std::integral_constant<int, LANES>(), nv);
  });
}
template <int V, int LANES, typename F>
void shape_one(const F& f) {
  f(std::integral_constant<int, V>(), std::integral_constant<int, LANES>(),
    std::integral_constant<int, 1>());
}
template <int V, bool GRAD, typename F>
bool with_shape(int64_t cols, int32_t dtype, const F& f) {
  const auto pieces = [&](auto lanes) {
    constexpr int L = decltype(lanes)::value;
    if constexpr (GRAD)
      shape_pieces<V, L, GradPieces<V, L>::kLeast, GradPieces<V, L>::kMost>(cols, f);
    else
      shape_pieces<V, L, L == 32 ? 2 : L == 64 && V == 4 ? 1 : 3, L == 1024 && V == 8 ? 3 : 4>(
          cols, f);
  };
  switch (GRAD ? grad_lanes(cols, dtype) : norm_lanes(cols, dtype)) {
    case 8:
      if (cols < V) shape_one<1, 8>(f);
      else shape_one<V, 8>(f);
      return true;
    case 16: shape_one<V, 16>(f); return true;
    case 32:
      if (cols <= 32 * V) shape_one<V, 32>(f);
      else if constexpr (V == 8 && !GRAD) pieces(std::integral_constant<int, 32>());
      return true;
    case 64: pieces(std::integral_constant<int, 64>()); return true;
    case 128:       // bfloat16 rows of the backward pass go from 64 to 256
      if constexpr (V == 4 || !GRAD) pieces(std::integral_constant<int, 128>());
      return true;
    case 256: pieces(std::integral_constant<int, 256>()); return true;
    case 512: pieces(std::integral_constant<int, 512>()); return true;
    case 1024: pieces(std::integral_constant<int, 1024>()); return true;
    default: return false;
  }
}

template <typename T, typename TW>
hipError_t rms(const RmsArgs& a, hipStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  const bool once = (a.R ? 4 : 2) * a.rows * a.cols * (int64_t)sizeof(T) > kCacheBytes;
  const bool held = with_shape<V, false>(a.cols, a.x_dtype, [&](auto v, auto lanes, auto nv) {
    constexpr int VV = decltype(v)::value, L = decltype(lanes)::value, N = decltype(nv)::value;
    constexpr int THREADS = L > 64 ? L : 256, GROUPS = THREADS / L;
    const dim3 grid((unsigned)std::min<int64_t>((a.rows + GROUPS - 1) / GROUPS, kMaxBlocks));
    if (a.scales)
      hipLaunchKernelGGL((k_rms<T, TW, VV, L, N, true>), grid, dim3(THREADS), 0, s, a, once);
    else
      hipLaunchKernelGGL((k_rms<T, TW, VV, L, N, false>), grid, dim3(THREADS), 0, s, a, once);
  });
  if (!held) {
    const bool in_place = a.Y == a.X || (a.R && (a.H == a.X || a.H == a.R));
    const int64_t share =
        in_place ? 1 : std::max<int64_t>(1, std::min(256 / a.rows, a.cols / 8192));
    hipLaunchKernelGGL((k_rms_long<T, TW, V>),
                       dim3((unsigned)std::min(a.rows, kMaxBlocks), (unsigned)share),
                       dim3(kRmsThreads), 0, s, a);
  }
  return hipGetLastError();
}

// As in the layer norm: one launch for few rows.
bool rms_few(int64_t rows, int64_t cols) {
  return rows > 0 && rows <= 2048 && rows * cols <= ((int64_t)1 << 22) && cols <= 16384;
}
// Blocks whose partial sums are joined.
int64_t rms_blocks(int64_t rows, int64_t cols, int32_t dtype) {
  const int lanes = grad_lanes(cols, dtype);
  if (lanes == 0)     // runs of rows: 16 waves a CU, at least 8 rows a wave
    return std::min((rows + 7) / 8, std::max<int64_t>(1, 4096 * kRmsCols / cols));
  const int groups = lanes > 512 ? 1 : 512 / lanes;
  return std::min<int64_t>((rows + groups - 1) / groups, lanes > 512 ? 256 : kGradBlocks);
}
size_t rms_part_bytes(int64_t blocks, int64_t cols) {
  return ((size_t)blocks * cols * 4 + 255) / 256 * 256;
}

template <typename T, typename TW, typename TO>
hipError_t rms_grad_few(const RmsGradArgs& a, hipStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  with_shape<V, true>(a.cols, a.x_dtype, [&](auto v, auto lanes, auto nv) {
    constexpr int VV = decltype(v)::value, L = decltype(lanes)::value, N = decltype(nv)::value;
    constexpr int THREADS = L > 512 ? L : 512, GROUPS = THREADS / L;
    const int row_blocks = a.dX ? (int)((a.rows + GROUPS - 1) / GROUPS) : 0;
    const int col_blocks = a.dgamma ? (int)((a.cols + 15) / 16) : 0;
    const auto go = [&](int rows, int cols) {
      if (rows + cols > 0)
        hipLaunchKernelGGL((k_rms_grad_few<T, TW, TO, VV, L, N>), dim3((unsigned)(rows + cols)),
                           dim3(THREADS), 0, s, a, rows);
    };
    if (a.dX == a.dY) {
      go(0, col_blocks);
      go(row_blocks, 0);
    } else {
      go(row_blocks, col_blocks);
    }
  });
  return hipGetLastError();
}

template <typename TO>
hipError_t rms_join(const RmsGradArgs& a, const float* part, int64_t blocks, hipStream_t s) {
  if (blocks <= 16)
    hipLaunchKernelGGL(k_rms_join_few<TO>, dim3((unsigned)((a.cols + 255) / 256)), dim3(256), 0, s,
                       part, (int)blocks, (int)a.cols, (TO*)a.dgamma, a.accumulate);
  else
    hipLaunchKernelGGL(k_rms_join<TO>, dim3((unsigned)((a.cols + 15) / 16)), dim3(1024), 0, s, part,
                       (int)blocks, (int)a.cols, (TO*)a.dgamma, a.accumulate);
  return hipGetLastError();
}

template <typename T, typename TW>
hipError_t rms_grad(const RmsGradArgs& a, hipStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  if (rms_few(a.rows, a.cols))
    return a.dw_dtype == SM_BF16 ? rms_grad_few<T, TW, bf16_t>(a, s)
                                 : rms_grad_few<T, TW, float>(a, s);
  const int64_t blocks = rms_blocks(a.rows, a.cols, a.x_dtype);
  float* part = a.dgamma ? (float*)a.ws : nullptr;
  if (a.rows > 0) {
    const bool once = 4 * a.rows * a.cols * (int64_t)sizeof(T) > kCacheBytes;
    const bool held = with_shape<V, true>(a.cols, a.x_dtype, [&](auto v, auto lanes, auto nv) {
      constexpr int VV = decltype(v)::value, L = decltype(lanes)::value, N = decltype(nv)::value;
      hipLaunchKernelGGL((k_rms_grad<T, TW, VV, L, N>), dim3((unsigned)blocks),
                         dim3(L > 512 ? L : 512), 0, s, a, once, part);
    });
    if (!held) {
      // all of dY and H is read before dX, which may be dY, is written
      const int64_t run = (a.rows + blocks - 1) / blocks;
      float* share = a.dX ? (float*)((char*)a.ws + rms_part_bytes(blocks, a.cols)) : nullptr;
      hipLaunchKernelGGL((k_rms_long_sums<T, TW, V>),
                         dim3((unsigned)((a.cols + 4 * kRmsCols - 1) / (4 * kRmsCols)),
                              (unsigned)blocks),
                         dim3(256), 0, s, a, run, part, share);
      if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
      if (a.dX)
        hipLaunchKernelGGL((k_rms_grad_long<T, TW, V>),
                           dim3((unsigned)((a.cols + 4095) / 4096),
                                (unsigned)std::min<int64_t>(a.rows, 65535)),
                           dim3(256), 0, s, a, share);
    }
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (!a.dgamma || (a.rows == 0 && a.accumulate)) return hipSuccess;
  return a.dw_dtype == SM_BF16 ? rms_join<bf16_t>(a, part, blocks, s)
                               : rms_join<float>(a, part, blocks, s);
}

}  // namespace

size_t rms_grad_workspace(int64_t rows, int64_t cols) {
  if (rms_few(rows, cols)) return 0;
  const int64_t blocks =
      std::max(rms_blocks(rows, cols, SM_F32), rms_blocks(rows, cols, SM_BF16));
  const int64_t waves = (cols + kRmsCols - 1) / kRmsCols;
  return rms_part_bytes(blocks, cols) +
         (grad_lanes(cols, SM_F32) ? 0 : (size_t)(rows * waves) * 4);
}

hipError_t launch_rms(const RmsArgs& a, hipStream_t s) {
  if (a.x_dtype == SM_BF16)
    return a.w_dtype == SM_BF16 ? rms<bf16_t, bf16_t>(a, s) : rms<bf16_t, float>(a, s);
  return a.w_dtype == SM_BF16 ? rms<float, bf16_t>(a, s) : rms<float, float>(a, s);
}

hipError_t launch_rms_grad(const RmsGradArgs& a, hipStream_t s) {
  if (a.x_dtype == SM_BF16)
    return a.w_dtype == SM_BF16 ? rms_grad<bf16_t, bf16_t>(a, s) : rms_grad<bf16_t, float>(a, s);
  return a.w_dtype == SM_BF16 ? rms_grad<float, bf16_t>(a, s) : rms_grad<float, float>(a, s);
}

}  // namespace sm
