// Products with few rows of activations (single tokens of a few sequences): out[n]
// [m] = sum over k of W(m, k) x(n, k), n <= 16, W with k along its rows.  Bound by
// reading W once.
//
// A wave multiplies 16 rows of W by all rows of x, with the weights' 16-byte
// pieces going from memory to registers in the layout that the matrix
// instructions take (lane l holds a piece of row l % 16; which k an instruction
// sums does not matter as long as x has the same), 8 pieces a matrix in flight.
// WK waves share a group's k and meet in LDS, in a fixed order.
#pragma once

#include "sm_lds.h"
#include "sm_rows.h"

namespace sm {

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

// NA matrices of the same shape go side by side (w0, w1).  Epi gets, for rows m0 ..
// m0 + 15 of W, acc[matrix][i] of row m0 + 4 (lane / 16) + i and row lane % 16 of x.
template <typename T, int NA, int WK, class Epi>
__global__ __launch_bounds__(512) void k_few(const T* w0, const T* w1, int64_t ldw, int m,
                                             const T* x, int64_t xs, int n, const int32_t* count,
                                             int k, typename Epi::Args ea) {
  constexpr int V = 16 / (int)sizeof(T), STEP = 4 * V, U = 8, PER = 8 / WK;
  __shared__ f32x4_t sh[WK > 1 ? 2 : 1][WK > 1 ? NA : 1][WK > 1 ? WK : 1][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = wave % WK;
  if (count) n = *count;
  if (n == 0) return;
  const int xr = (lane & 15) < n ? lane & 15 : n - 1;
  const T* xrow = x + (int64_t)xr * xs;
  const int steps = (k + STEP - 1) / STEP, per = (steps + WK - 1) / WK;
  const int s0 = part * per, s1 = s0 + per < steps ? s0 + per : steps;
  const int groups = (m + 15) / 16;
  Epi epi(ea, lane, n);
  int turn = 0;
  for (int g = blockIdx.x * PER + wave / WK; g < groups; g += gridDim.x * PER) {
    const int row = g * 16 + (lane & 15);
    const int64_t at = (int64_t)(row < m ? row : m - 1) * ldw;
    f32x4_t acc[NA];
#pragma unroll
    for (int a = 0; a < NA; ++a) acc[a] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    int s = s0;
    for (; s + U <= s1 && (s + U) * STEP <= k; s += U) {
      u32x4_t w[NA][U], xv[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = (s + u) * STEP + (lane >> 4) * V;
#pragma unroll
        for (int a = 0; a < NA; ++a) {
          Piece<T, V> p;
          p.template load<true>((a ? w1 : w0) + at + c);
          w[a][u] = u32x4_t{p.w[0], p.w[1], p.w[2], p.w[3]};
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        Piece<T, V> p;
        p.load(xrow + (s + u) * STEP + (lane >> 4) * V);
        xv[u] = u32x4_t{p.w[0], p.w[1], p.w[2], p.w[3]};
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int a = 0; a < NA; ++a) acc[a] = few_multiply<T>(w[a][u], xv[u], acc[a]);
    }
    for (; s < s1; ++s) {
      const int c = s * STEP + (lane >> 4) * V;
      const u32x4_t xv = few_piece(xrow, c, k);
#pragma unroll
      for (int a = 0; a < NA; ++a)
        acc[a] = few_multiply<T>(few_piece((a ? w1 : w0) + at, c, k), xv, acc[a]);
    }
    if constexpr (WK > 1) {      // (PER = 1: the block's waves go through the same groups)
      static_assert(WK == 1 || WK == 8, "waves of a group");
#pragma unroll
      for (int a = 0; a < NA; ++a) sh[turn][a][part][lane] = acc[a];
      __syncthreads();
      if (part == 0) {
#pragma unroll
        for (int a = 0; a < NA; ++a)
#pragma unroll
          for (int q = 1; q < WK; ++q) acc[a] += sh[turn][a][q][lane];
        epi.group(g * 16, m, acc);
      }
      turn ^= 1;
    } else {
      epi.group(g * 16, m, acc);
    }
  }
  epi.finish(blockIdx.x * 8 + wave);
}

}  // namespace sm
