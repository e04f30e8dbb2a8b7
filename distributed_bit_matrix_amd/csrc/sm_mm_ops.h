// Epilogues, operand copies and launches shared by the feed-forward and loss
// operators.
#pragma once

#include "sm_mm.h"
#include "sm_rows.h"

namespace sm {

// Three bfloat16 values whose sum is f to 24 bits.  Each is taken of what the
// others leave, which is exact; a value that is not finite is in the first.
__device__ __forceinline__ void split3(float f, bf16_t (&p)[3]) {
  p[0] = f32_to_bf16(f);
  const float hi = bf16_to_f32(p[0]);
  const float r = __builtin_isfinite(hi) ? f - hi : 0.f;
  p[1] = f32_to_bf16(r);
  p[2] = f32_to_bf16(r - bf16_to_f32(p[1]));
}
// Four neighbouring entries to P planes, `plane` entries apart; 8-byte aligned.
template <int P>
__device__ __forceinline__ void store_planes(bf16_t* p, int64_t plane, const float (&v)[4]) {
  if constexpr (P == 1) {
    *reinterpret_cast<u32x2_t*>(p) = u32x2_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
  } else {
    bf16_t t[4][3];
#pragma unroll
    for (int k = 0; k < 4; ++k) split3(v[k], t[k]);
#pragma unroll
    for (int q = 0; q < 3; ++q)
      *reinterpret_cast<u32x2_t*>(p + q * plane) =
          u32x2_t{(uint32_t)t[0][q] | ((uint32_t)t[1][q] << 16),
                  (uint32_t)t[2][q] | ((uint32_t)t[3][q] << 16)};
  }
}

// The product itself: to an array of a caller's type, or (parts) to float32
// sums of a split, which a later launch joins.
struct MmOut {
  void* p;
  int64_t ld;
  int64_t split_step;      // elements from one split's sums to the next
  int32_t dtype, add;      // add: to what is there (float32)
};
struct EpiStore {
  struct Args {
    MmOut out[kMaxJobs];
  };
  template <int TI, int TJ>
  static __device__ __forceinline__ void run(const Args& e, const MmPlace& at,
                                             const f32x4_t (&acc)[TI][TJ]) {
    const MmOut o = e.out[at.job];
    const int mc = at.m0 + 4 * (at.lane >> 4), nc = at.n0 + (at.lane & 15);
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const int n = nc + 16 * j;
      if (n >= at.n) continue;
      const int64_t row = (int64_t)n * o.ld + at.split * o.split_step;
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        const int m = mc + 16 * i;
        if (m >= at.m) continue;
        float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
        const int here = at.m - m;
        if (o.dtype == SM_F32) {
          float* p = static_cast<float*>(o.p) + row + m;
          if (here >= 4) {
            if (o.add) {
              const u32x4_a4 t = *reinterpret_cast<const u32x4_a4*>(p);
#pragma unroll
              for (int k = 0; k < 4; ++k) v[k] += __uint_as_float(t[k]);
            }
            store_vec<4>(p, v);
          } else {
            for (int k = 0; k < here; ++k) p[k] = (o.add ? p[k] : 0.f) + v[k];
          }
        } else {
          bf16_t* p = static_cast<bf16_t*>(o.p) + row + m;
          if (here >= 4) store_vec<4>(p, v);
          else
            for (int k = 0; k < here; ++k) p[k] = f32_to_bf16(v[k]);
        }
      }
    }
  }
};

// Rows of a caller's matrix as `planes` bfloat16 planes of row length ld, its
// pad zero.  list, count: rows list[0 .. *count), or all where list is null.
struct PlanesArgs {
  const void* src;
  int64_t stride;
  int32_t dtype, planes;
  int64_t rows;
  int32_t cols, ld;
  const int32_t *list, *count;
  bf16_t* dst;
};
hipError_t launch_planes(const PlanesArgs& a, hipStream_t s);

// Sums of splits joined: out[r][c] = sum over s of part[s][at(r)][c] (plus what
// is there), at(r) = pos[r], or r where pos is null; a row whose pos is negative
// is zero.
struct JoinArgs {
  const float* part;
  int64_t split_step, part_ld;
  int32_t splits;
  const int32_t* pos;
  int64_t rows;
  int32_t cols, dtype, add;
  void* out;
  int64_t ld;
};
hipError_t launch_join(const JoinArgs& a, hipStream_t s);

hipError_t launch_zero(void* p, int32_t dtype, int64_t n, hipStream_t s);

// Whether a matrix can be an operand where it lies: rows of whole 16-byte
// pieces, and offsets within a tile of 31 bits.
inline bool operand_fits(const void* p, int32_t dtype, int64_t cols, int64_t stride) {
  return dtype == SM_BF16 && (uintptr_t)p % 16 == 0 && cols % 8 == 0 && stride % 8 == 0 &&
         stride <= ((int64_t)1 << 21);
}

// The pairs of planes of a float32 product: those whose products reach 2^-24 of
// the largest.  The small ones come first.
constexpr int kPairs[6][2] = {{2, 0}, {1, 1}, {0, 2}, {1, 0}, {0, 1}, {0, 0}};
// Adds the segments of one product to a job; planes: 1 or 3, a_plane and b_plane
// in bytes, a_at and b_at where the product's operands begin.
inline void add_segs(MmJob& j, int planes, int64_t a_plane, int64_t b_plane, int64_t a_at = 0,
                     int64_t b_at = 0) {
  for (int s = 0; s < (planes == 1 ? 1 : 6); ++s) {
    j.a_seg[j.segs] = a_at + (planes == 1 ? 0 : kPairs[s][0] * a_plane);
    j.b_seg[j.segs++] = b_at + (planes == 1 ? 0 : kPairs[s][1] * b_plane);
  }
}

constexpr int kCus = 256;
// Tiles of 256 x 256 where they fill the chip, or nearly; else 128 x 128.
inline bool wide_tiles(int64_t m, int64_t n) {
  return ((m + 255) / 256) * ((n + 255) / 256) >= 160;
}
// How many blocks share a tile's k: as many as fill the chip, each with 8 slabs
// at least.
inline int k_splits(int64_t m, int64_t n, int64_t slabs, bool wide) {
  const int t = wide ? 256 : 128;
  const int64_t tiles = ((m + t - 1) / t) * ((n + t - 1) / t);
  const int64_t want = (wide ? kCus : 2 * kCus) / std::max<int64_t>(1, tiles);
  return (int)std::max<int64_t>(1, std::min<int64_t>({want, slabs / 8, 16}));
}

// Launches the jobs of `a` (operands, extents, segments and splits are set).
template <bool AKM, bool BKM, bool PAIR, class Sh, class Epi>
hipError_t run_mm_as(MmArgs& a, const typename Epi::Args& e, hipStream_t s) {
  int64_t blocks = 0;
  for (int i = 0; i < a.jobs; ++i) {
    MmJob& j = a.job[i];
    const int tm = PAIR ? Sh::TM / 2 : Sh::TM;
    j.m_tiles = (j.m + tm - 1) / tm;
    j.n_tiles = (j.n + Sh::TN - 1) / Sh::TN;
    j.block0 = (int)blocks;
    blocks += (int64_t)j.m_tiles * j.n_tiles * j.splits;
  }
  if (blocks == 0) return hipSuccess;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  a.blocks = (int)blocks;
  hipLaunchKernelGGL((k_mm<AKM, BKM, PAIR, Sh, Epi>), dim3((unsigned)blocks),
                     dim3(64 * Sh::WAVES), 0, s, a, e);
  return hipGetLastError();
}
template <bool AKM, bool BKM, bool PAIR, class Epi>
hipError_t run_mm(MmArgs& a, const typename Epi::Args& e, bool wide, hipStream_t s) {
  return wide ? run_mm_as<AKM, BKM, PAIR, MmShape<256, 256, 2, 4>, Epi>(a, e, s)
              : run_mm_as<AKM, BKM, PAIR, MmShape<128, 128, 2, 2>, Epi>(a, e, s);
}

}  // namespace sm
