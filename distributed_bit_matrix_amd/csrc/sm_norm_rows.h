// How the norms hold a row: a group of LANES threads, NV pieces of 16 bytes each.
#pragma once

#include <algorithm>
#include <type_traits>

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

constexpr int64_t kMaxBlocks = 1 << 16;   // larger grids loop
constexpr int kGradBlocks = 512;          // two blocks of 512 threads a CU

inline int vec_of(int32_t dtype) { return dtype == SM_BF16 ? 8 : 4; }

// Threads a row, 0: too long for registers.  Rows shorter than a piece go
// entry by entry (8 threads).
//
// Forward: up to 4 pieces a thread, in as few threads as hold the row, so that
// few of them idle past its end: 12288 x 768 bfloat16 takes 9.1 us with 32 x 3
// pieces, 10.6 us with 64 x 2 (a quarter idle) and 12.7 us with 128 x 1.  Four
// pieces of bfloat16 in 1024 threads need more than their 128 registers: 2048 x
// 24576 takes 46 us from registers and 52 in k_norm_long, 2048 x 25000 83 and
// 54.
inline int norm_lanes(int64_t cols, int32_t dtype) {
  const int vec = vec_of(dtype);
  for (int lanes : {8, 16, 32})
    if (cols <= lanes * vec) return lanes;
  if (vec == 8 && cols <= 32 * 8 * 4) return 32;
  for (int lanes : {64, 128, 256, 512, 1024})
    if (cols <= (int64_t)lanes * vec * (lanes == 1024 && vec == 8 ? 3 : 4)) return lanes;
  return 0;
}
// Backward: a thread holds five values an entry.  16 entries a thread leave
// too few waves to cover the loads; 8 are better even where the row then takes
// several waves (16384 x 4096 bfloat16 78 against 83 us, 333 x 1001 float32
// 4.6 against 6.5 us) but for rows of one wave in bfloat16 (12288 x 768 14.8
// against 16.4 us).
inline int grad_lanes(int64_t cols, int32_t dtype) {
  const int vec = vec_of(dtype);
  for (int lanes : {8, 16, 32})
    if (cols <= lanes * vec) return lanes;
  if (cols <= (vec == 8 ? 1024 : 512)) return 64;
  for (int lanes : {64, 128, 256, 512, 1024})
    if (cols <= lanes * 8) return lanes;
  return cols <= 16384 ? 1024 : 0;
}

// Calls f with the number of pieces a thread as a constant, between LEAST and
// MOST, which are all that norm_lanes and grad_lanes leave for a group's width.
template <int LEAST, int MOST, typename F>
void with_pieces(int64_t nv, const F& f) {
  if constexpr (LEAST < MOST)
    if (nv > LEAST) return with_pieces<LEAST + 1, MOST>(nv, f);
  f(std::integral_constant<int, LEAST>());
}
template <int V, int LANES>
struct GradPieces {
  static constexpr int kLeast = LANES == 64 || V == 8 ? 1 : 2;
  static constexpr int kMost = LANES == 64 ? 2 : LANES == 1024 ? (V == 8 ? 2 : 4) : kLeast;
};

}  // namespace sm
