// Products with few rows of activations (single tokens of a few sequences): out[n]
// [m] = sum over k of W(m, k) x(n, k), n <= 16, W with k along its rows.  Bound by
// reading W once.
//
// A wave multiplies 16 rows of W by all rows of x, with the weights' 16-byte
// pieces going from memory to registers in the layout that the matrix
// instructions take (lane l holds a piece of row l % 16; which k an instruction
// sums does not matter as long as x has the same).  Many waves with 2 pieces a
// matrix each in flight: 4096 x 16384 bfloat16 27 us (5 TB/s; 8 pieces in half the
// waves 32, the next pieces fetched ahead in registers 78).  float32 goes through the
// float32 matrix instructions (busy for a quarter of the time): one row of a block of 4096 x
// 16384 108 + 68 us, 4.9 and 3.9 TB/s, which is slower as a call (184 us, 16 rows 217)
// than elementary operations (168, 172).
// WK waves share a group's k and meet in LDS, in a fixed order.
#pragma once

#include <algorithm>
#include <type_traits>

#include "sm_lds.h"
#include "sm_rows.h"

namespace sm {

// Rows up to which this is the form.  More in a wave do not pay: a block of 4096 x
// 16384 bfloat16, 32 rows a wave 132 us, 64 rows 196, the tiles 114 and 122.
constexpr int kFewRows = 16;

// 16 bytes of a row as they lie in memory; past the row's end zeros.
template <typename T>
__device__ __forceinline__ u32x4_t few_piece(const T* row, int k, int k_all) {
  constexpr int V = 16 / (int)sizeof(T);
  if (k + V <= k_all) {
    Piece<T, V> p;
    p.load(row + k);
    return u32x4_t{p.w[0], p.w[1], p.w[2], p.w[3]};
  }
  u32x4_t v = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < V; ++e) {
    if (k + e < k_all) {
      if constexpr (sizeof(T) == 4) v[e] = __float_as_uint(row[k + e]);
      else v[e / 2] |= (uint32_t)row[k + e] << (16 * (e & 1));
    }
  }
  return v;
}

template <typename T>
__device__ __forceinline__ f32x4_t few_multiply(u32x4_t w, u32x4_t x, f32x4_t acc) {
  if constexpr (sizeof(T) == 2) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w),
                                                   __builtin_bit_cast(bf16x8_t, x), acc, 0, 0, 0);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w[e]), __uint_as_float(x[e]), acc,
                                                 0, 0, 0);
    return acc;
  }
}

// A lane's share of one step of x: as many values as a 16-byte piece of W has.
template <typename T, typename X>
struct FewX {                  // x in W's type
  u32x4_t w;
  __device__ __forceinline__ void zero() { w = u32x4_t{0, 0, 0, 0}; }
  __device__ __forceinline__ void load(const X* at) {
    Piece<X, 16 / (int)sizeof(X)> p;
    p.load(at);
    w = u32x4_t{p.w[0], p.w[1], p.w[2], p.w[3]};
  }
  __device__ __forceinline__ void edge(const X* row, int k, int k_all) {
    w = few_piece(row, k, k_all);
  }
  __device__ __forceinline__ f32x4_t multiply(u32x4_t a, f32x4_t acc) const {
    return few_multiply<T>(a, w, acc);
  }
};

// x in float32 beside bfloat16 weights: x = hi + lo of two bfloat16, which leaves
// 2^-18 of a value, and two instructions a piece.
template <>
struct FewX<bf16_t, float> {
  u32x4_t w[2];
  __device__ __forceinline__ void zero() { w[0] = w[1] = u32x4_t{0, 0, 0, 0}; }
  __device__ __forceinline__ void load(const float* at) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      Piece<float, 4> p;
      p.load(at + 4 * i);
      w[i] = u32x4_t{p.w[0], p.w[1], p.w[2], p.w[3]};
    }
  }
  __device__ __forceinline__ void edge(const float* row, int k, int k_all) {
    w[0] = few_piece(row, k, k_all);
    w[1] = few_piece(row, k + 4, k_all);
  }
  __device__ __forceinline__ f32x4_t multiply(u32x4_t a, f32x4_t acc) const {
    u32x4_t hi, lo;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float v0 = __uint_as_float(w[i / 2][2 * (i & 1)]);
      const float v1 = __uint_as_float(w[i / 2][2 * (i & 1) + 1]);
      hi[i] = pack_bf16(first_plane(v0), first_plane(v1));
      const float h0 = __uint_as_float(hi[i] << 16), h1 = __uint_as_float(hi[i] & 0xffff0000u);
      lo[i] = pack_bf16(__builtin_isfinite(h0) ? v0 - h0 : 0.f,
                        __builtin_isfinite(h1) ? v1 - h1 : 0.f);
    }
    return few_multiply<bf16_t>(a, hi, few_multiply<bf16_t>(a, lo, acc));
  }
};

// Waves of a block, and how many of them share a group's k: as many as make 24
// waves a CU, each with 2 steps at least.
constexpr int few_waves(int wk) { return wk > 8 ? wk : 8; }
inline int few_share(int64_t m, int64_t k, int step) {
  const int64_t groups = (m + 15) / 16, steps = (k + step - 1) / step;
  int wk = 1;
  while (wk < 16 && groups * wk < 24 * 256 && steps >= 4 * wk) wk *= 2;
  return wk;
}

// NA matrices of the same shape go side by side (w0, w1).  Epi gets, for rows m0 ..
// m0 + 15 of W, acc[matrix][i] of row m0 + 4 (lane / 16) + i and row lane % 16 of x.
template <typename T, typename X, int NA, int WK, class Epi>
__global__ __launch_bounds__(64 * few_waves(WK)) void k_few(const T* w0, const T* w1, int64_t ldw,
                                                            int m, const X* x, int64_t xs, int n,
                                                            int k, bool once,
                                                            typename Epi::Args ea) {
  constexpr int V = 16 / (int)sizeof(T), STEP = 4 * V, U = 2, PER = few_waves(WK) / WK;
  __shared__ f32x4_t sh[WK > 1 ? 2 : 1][WK > 1 ? NA : 1][WK > 1 ? PER * WK : 1][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = wave % WK, mine = wave / WK;
  const int xr = (lane & 15) < n ? lane & 15 : n - 1;
  const X* xrow = x + (int64_t)xr * xs;
  const int steps = (k + STEP - 1) / STEP, per = (steps + WK - 1) / WK;
  const int s0 = part * per, s1 = s0 + per < steps ? s0 + per : steps;
  const int groups = (m + 15) / 16;
  Epi epi(ea, lane, n);
  int turn = 0;
  // (a block's waves go through the same turns: they meet in barriers)
  for (int g0 = blockIdx.x * PER; g0 < groups; g0 += gridDim.x * PER) {
    const int g = g0 + mine < groups ? g0 + mine : groups - 1;
    const int row = g * 16 + (lane & 15);
    const int64_t at = (int64_t)(row < m ? row : m - 1) * ldw;
    f32x4_t acc[NA];
#pragma unroll
    for (int a = 0; a < NA; ++a) acc[a] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    int s = s0;
    for (; s + U <= s1 && (s + U) * STEP <= k; s += U) {
      u32x4_t w[NA][U];
      FewX<T, X> xv[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = (s + u) * STEP + (lane >> 4) * V;
#pragma unroll
        for (int a = 0; a < NA; ++a) {
          Piece<T, V> p;
          if (once) p.template load<true>((a ? w1 : w0) + at + c);
          else p.load((a ? w1 : w0) + at + c);
          w[a][u] = u32x4_t{p.w[0], p.w[1], p.w[2], p.w[3]};
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) xv[u].load(xrow + (s + u) * STEP + (lane >> 4) * V);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int a = 0; a < NA; ++a) acc[a] = xv[u].multiply(w[a][u], acc[a]);
    }
    if (s < s1) {
      // what is left, in one go: pieces past the end (of the share, or of the row)
      // are loaded from the row's beginning and count as zeros
      u32x4_t w[NA][U];
      FewX<T, X> xv[U];
      const u32x4_t zero = {0, 0, 0, 0};
      if (V <= k) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int c = (s + u) * STEP + (lane >> 4) * V;
          const int from = s + u < s1 && c + V <= k ? c : 0;
          Piece<T, V> p;
#pragma unroll
          for (int a = 0; a < NA; ++a) {
            p.load((a ? w1 : w0) + at + from);
            w[a][u] = u32x4_t{p.w[0], p.w[1], p.w[2], p.w[3]};
          }
          xv[u].load(xrow + from);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int c = (s + u) * STEP + (lane >> 4) * V;
          const bool in = s + u < s1 && c + V <= k;
          if (!in) xv[u].zero();
#pragma unroll
          for (int a = 0; a < NA; ++a) acc[a] = xv[u].multiply(in ? w[a][u] : zero, acc[a]);
        }
      }
      // a row's last, shorter piece
      for (; s < s1; ++s) {
        if (s + 1 < steps || k % V == 0) continue;
        const int c = s * STEP + (lane >> 4) * V;
        const bool in = c < k && c + V > k;
        FewX<T, X> xe;
        xe.zero();
        if (in) xe.edge(xrow, c, k);
#pragma unroll
        for (int a = 0; a < NA; ++a)
          acc[a] = xe.multiply(in ? few_piece((a ? w1 : w0) + at, c, k) : zero, acc[a]);
      }
    }
    if constexpr (WK > 1) {
#pragma unroll
      for (int a = 0; a < NA; ++a) sh[turn][a][wave][lane] = acc[a];
      __syncthreads();
      if (part == 0 && g0 + mine < groups) {
#pragma unroll
        for (int a = 0; a < NA; ++a)
#pragma unroll
          for (int q = 1; q < WK; ++q) acc[a] += sh[turn][a][wave + q][lane];
        epi.group(g * 16, m, acc);
      }
      turn ^= 1;
    } else if (g0 + mine < groups) {
      epi.group(g * 16, m, acc);
    }
  }
  if (part == 0) epi.finish(blockIdx.x * PER + mine);
}

// Blocks of a launch: as many as there are groups for, up to 8192 waves (32 a CU).
inline int64_t few_blocks(int64_t m, int wk) {
  const int waves = few_waves(wk), per = waves / wk;
  return std::min<int64_t>(((m + 15) / 16 + per - 1) / per, 8192 / waves);
}
// Numbers that `finish` gets are below this.
template <typename T>
int few_strips(int64_t m, int64_t k) {
  const int wk = few_share(m, k, 64 / (int)sizeof(T));
  return (int)few_blocks(m, wk) * (few_waves(wk) / wk);
}

template <typename T, typename X, int NA, class Epi>
hipError_t launch_few(const T* w0, const T* w1, int64_t ldw, int64_t m, const X* x, int64_t xs,
                      int64_t n, int64_t k, const typename Epi::Args& ea, hipStream_t s) {
  const bool once = NA * m * k * (int64_t)sizeof(T) > kCacheBytes;
  const auto go = [&](auto wk) {
    constexpr int WK = decltype(wk)::value;
    hipLaunchKernelGGL((k_few<T, X, NA, WK, Epi>), dim3((unsigned)few_blocks(m, WK)),
                       dim3(64 * few_waves(WK)), 0, s, w0, w1, ldw, (int)m, x, xs, (int)n, (int)k,
                       once, ea);
    return hipGetLastError();
  };
  switch (few_share(m, k, 64 / (int)sizeof(T))) {
    case 1: return go(std::integral_constant<int, 1>());
    case 2: return go(std::integral_constant<int, 2>());
    case 4: return go(std::integral_constant<int, 4>());
    case 8: return go(std::integral_constant<int, 8>());
    default: return go(std::integral_constant<int, 16>());
  }
}

}  // namespace sm
