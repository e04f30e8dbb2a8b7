// Products of float32 weights with up to 512 rows: sums[split][n][m] = sum over a
// share of k of W(m, k) x(n, k), W with either index along its rows.  The tiles of
// sm_mm.h want bfloat16 planes of both operands in memory, which for weights that
// one tile of rows reads once costs several times their reading.  Here W is read
// once (for every 128 rows of x), as float32.
//
// A wave takes 32 rows of W from memory to registers, a step of 64 k ahead, and
// splits them into three bfloat16 planes there (truncated, so that their sum is W
// itself); x has its planes in memory, and a block's 8 waves share a step of them in
// LDS, in two turns.  The six products of planes are those of sm_mm.h.  Bound by
// reading W, one step in flight: 17 rows, two matrices of 16384 x 4096 with k along rows
// 132 us (4.1 TB/s), with m along rows 116 (4.6); 126047 x 2436 with k along rows 331,
// and 381 in the backward pass (3.7, 3.2), with m 281 (4.4); 128 rows by the matrix units
// as well.  (Each wave loading x for itself from the caches: 17 rows of the first's block
// 296 us instead of 220, 128 rows 861 instead of 331.)
#pragma once

#include "sm_mm_ops.h"

namespace sm {

constexpr int kThinTile = 256;            // rows of W a block: 32 a wave
constexpr int kThinStep = 64;             // k

struct ThinArgs {
  const float* w[2];                      // matrices of one shape, rows of ldw
  const bf16_t* x[2];                     // of each: [3 planes][n][xs], xs in whole steps
  float* sums[2];                         // [split][n][m rounded up to 4] of each
  int64_t ldw, xs, plane;
  int32_t m, n, k, splits;
  int32_t mats;                           // matrices
  bool once;                              // W is larger than the caches
};

__device__ __forceinline__ void thin_split(const u32x4_t (&v)[2], u32x4_t (&p)[3]) {
  constexpr uint32_t kHigh = 0xFFFF0000u, kPick = 0x07060302u;   // the two high halves
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t a = v[i / 2][2 * (i & 1)], b = v[i / 2][2 * (i & 1) + 1];
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      p[q][i] = __builtin_amdgcn_perm(b, a, kPick);
      a = __float_as_uint(__uint_as_float(a) - __uint_as_float(a & kHigh));
      b = __float_as_uint(__uint_as_float(b) - __uint_as_float(b & kHigh));
    }
  }
}

// NB groups of 16 rows of x.  KM: a row of W is a k.  A lane then loads two
// neighbours of each of its 8 k, one for each of its wave's groups of 16, so these
// alternate.  In LDS a plane's row has 128 bytes, its 16-byte pieces
// in an order that its number decides, so that 16 rows of a piece lie in distinct
// banks.  Grid: tiles of W, splits, matrices times tiles of x.
template <int NB, bool KM>
__global__ __launch_bounds__(512) void k_thin(ThinArgs a) {
  constexpr int PIECES = 3 * NB * 16 * 8, MINE = (PIECES + 511) / 512;
  __shared__ u32x4_t sh[2][PIECES];
  const int lane = threadIdx.x & 63, c0 = (lane >> 4) * 8;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m0 = blockIdx.x * kThinTile + wave * 32, mat = blockIdx.z % a.mats;
  const int n0 = (int)(blockIdx.z / a.mats) * NB * 16, n = a.n - n0;
  const int steps = (a.k + kThinStep - 1) / kThinStep, per = (steps + a.splits - 1) / a.splits;
  const int s0 = (int)blockIdx.y * per, end = s0 + per < steps ? s0 + per : steps;
  // KM: a lane's pair of m; one that would pass the end is the last pair, and its
  // second is the first group's.  Nothing branches about these loads or selects from
  // them before they are used: each would wait.
  const int pair = m0 + 2 * (lane & 15);
  const bool shifted = KM && pair > a.m - 2;
  const float* wr[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = m0 + 16 * i + (lane & 15);
    wr[i] = KM ? a.w[mat] + (shifted ? a.m - 2 : pair)
               : a.w[mat] + (int64_t)(row < a.m ? row : a.m - 1) * a.ldw;
  }
  // a thread's pieces of x: where from, where to, and which k of a step
  const bf16_t* from[MINE];
  int to[MINE], kx[MINE];
#pragma unroll
  for (int j = 0; j < MINE; ++j) {
    const int i = threadIdx.x + 512 * j, p = i & 7, r = i >> 3 & (NB * 16 - 1);
    const int q = i / (NB * 128);
    from[j] = a.x[mat] + q * a.plane + (int64_t)(n0 + (r < n ? r : n - 1)) * a.xs + 8 * p;
    to[j] = i < PIECES ? (q * NB * 16 + r) * 8 + (p ^ (r & 7)) : -1;
    kx[j] = 8 * p;
  }
  const auto load_x = [&](u32x4_t (&v)[MINE], int s) SM_INLINE {
#pragma unroll
    for (int j = 0; j < MINE; ++j) {
      v[j] = u32x4_t{0, 0, 0, 0};
      if (to[j] >= 0 && s * kThinStep + kx[j] < a.k)
        v[j] = *reinterpret_cast<const u32x4_t*>(from[j] + s * kThinStep);
    }
  };
  const auto store_x = [&](const u32x4_t (&v)[MINE], int turn) SM_INLINE {
#pragma unroll
    for (int j = 0; j < MINE; ++j)
      if (to[j] >= 0) sh[turn][to[j]] = v[j];
  };
  const auto load_w = [&](u32x4_t (&w)[2][2][2], int s) SM_INLINE {   // [half step][rows][piece]
    const bool whole = (s + 1) * kThinStep <= a.k;
    if constexpr (KM) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int c = s * kThinStep + 32 * h + c0 + j;
          // (past k the last row, where x is zero)
          const u32x2_a4* from =
              reinterpret_cast<const u32x2_a4*>(wr[0] + (int64_t)(c < a.k ? c : a.k - 1) * a.ldw);
          const u32x2_a4 t = a.once ? __builtin_nontemporal_load(from) : *from;
          w[h][0][j / 4][j % 4] = t[0];
          w[h][1][j / 4][j % 4] = t[1];
        }
      return;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const int c = s * kThinStep + 32 * h + c0 + 4 * p;
          if (whole) {
            Piece<float, 4> t;
            if (a.once) t.template load<true>(wr[i] + c);
            else t.load(wr[i] + c);
            w[h][i][p] = u32x4_t{t.w[0], t.w[1], t.w[2], t.w[3]};
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[h][i][p][e] = c + e < a.k ? __float_as_uint(wr[i][c + e]) : 0u;
          }
        }
  };
  f32x4_t acc[NB][2];
#pragma unroll
  for (int b = 0; b < NB; ++b) acc[b][0] = acc[b][1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  u32x4_t w[2][2][2];
  if (s0 < end) {
    u32x4_t v[MINE];
    load_w(w, s0);
    load_x(v, s0);
    store_x(v, 0);
  }
  __syncthreads();
  for (int s = s0, turn = 0; s < end; ++s, turn ^= 1) {
    u32x4_t next[2][2][2], v[MINE];
    if (s + 1 < end) {
      load_x(v, s + 1);
      load_w(next, s + 1);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u32x4_t p[2][3];
      if (KM && shifted) w[h][0][0] = w[h][1][0], w[h][0][1] = w[h][1][1];
      thin_split(w[h][0], p[0]);
      thin_split(w[h][1], p[1]);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        bf16x8_t xv[3];
#pragma unroll
        for (int q = 0; q < 3; ++q) {
          const int r = 16 * b + (lane & 15);
          xv[q] = __builtin_bit_cast(
              bf16x8_t, sh[turn][(q * NB * 16 + r) * 8 + ((4 * h + (lane >> 4)) ^ (r & 7))]);
        }
#pragma unroll
        for (int q = 0; q < 6; ++q) {
          const int pw = kPairCode >> (4 * q) & 3, px = kPairCode >> (4 * q + 2) & 3;
#pragma unroll
          for (int i = 0; i < 2; ++i)
            acc[b][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(bf16x8_t, p[i][pw]), xv[px], acc[b][i], 0, 0, 0);
        }
      }
    }
    if (s + 1 < end) {
      store_x(v, turn ^ 1);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int q = 0; q < 2; ++q) w[h][i][q] = next[h][i][q];
    }
    __syncthreads();
  }
  // a lane has 4 neighbouring rows of W of a row of x
  const int64_t ld = (a.m + 3) & ~3;
  float* out = a.sums[mat] + ((int64_t)blockIdx.y * a.n + n0) * ld;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int r = 16 * b + (lane & 15);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int f = m0 + (KM ? 8 * (lane >> 4) + 4 * i : 16 * i + 4 * (lane >> 4));
      f32x4_t v = acc[b][i];
      if constexpr (KM)
        v = f32x4_t{acc[b][0][2 * i], acc[b][1][2 * i], acc[b][0][2 * i + 1],
                    acc[b][1][2 * i + 1]};
      if (r < n && f < a.m) *reinterpret_cast<f32x4_t*>(out + r * ld + f) = v;
    }
  }
}

// Whether this is the form, for `mats` matrices of m times k.  Microseconds with the
// tiles and here, forward: 2^20 values (1024 x 1000) 128 rows 34, 40; 2^22 (768 x 2048,
// three) 128 rows 56, 51, 384 rows 67, 70; 2^25 (768 x 50257) 17 rows 179, 52, 512
// rows 318, 282; 2^28 (2436 x 126047) 17 rows 1350, 353, 512 rows 2222, 1946.
// Backward it is the form of the products with the weights, from one row on: 2^22
// values 1 row 59, 47, 64 rows 60, 60, 128 rows 61, 76; 2^23 (1000 x 10007) 64 rows 105,
// 103, 128 rows 112, 134; 2^25 17 rows 452, 172, 128 rows 482, 293; 2^28 17 rows 2436,
// 1068, 128 rows 2871, 1615.  Elementary operations (float32 library products, and h
// through memory) are faster where a block's weights are large and its rows few: 4096 x
// 16384, 17 rows 179 us and here 216, 64 rows 260 and 261, 128 rows 470 and 353; 2048 x
// 8192, 128 rows 131 and 157; gradients of the first, 1 row 477 and 506, 17 rows 548 and
// 525.
inline bool thin_form(int64_t rows, int64_t m, int64_t k, int mats, int32_t dtype,
                      bool backward) {
  const int64_t values = mats * m * k;
  if (dtype != SM_F32 || m < 2 || k < 2) return false;
  if (backward) return rows <= 128 && values >= (rows <= 64 ? 1 << 22 : 1 << 24);
  return rows > 16 && rows <= 512 && values >= (rows <= 128 ? 1 << 21 : 1 << 24);
}
// How many blocks share a tile's k: two blocks a CU, each with two steps at least, and
// sums that stay small beside the weights.
inline int thin_splits(int64_t m, int64_t n, int64_t k, int mats) {
  const int64_t tiles = mats * ((m + kThinTile - 1) / kThinTile) * ((n + 127) / 128);
  const int64_t steps = (k + kThinStep - 1) / kThinStep;
  return (int)std::max<int64_t>(1, std::min({2 * kCus / tiles, steps / 2, (int64_t)64}));
}
template <bool KM>
hipError_t launch_thin(const ThinArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.m + kThinTile - 1) / kThinTile), (unsigned)a.splits,
                  (unsigned)(a.mats * ((a.n + 127) / 128)));
  const int nb = (a.n + 15) / 16;
  if (nb <= 2) hipLaunchKernelGGL((k_thin<2, KM>), grid, dim3(512), 0, s, a);
  else if (nb <= 4) hipLaunchKernelGGL((k_thin<4, KM>), grid, dim3(512), 0, s, a);
  else hipLaunchKernelGGL((k_thin<8, KM>), grid, dim3(512), 0, s, a);
  return hipGetLastError();
}

}  // namespace sm
