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
  template <typename T, bool WHOLE, bool ADD, int TI, int TJ>
  static __device__ __forceinline__ void store(T* p, int64_t ld, const MmPlace& at,
                                               const f32x4_t (&acc)[TI][TJ]) {
    const int mc = at.m0 + 4 * (at.lane >> 4), nc = at.n0 + (at.lane & 15);
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      if (!WHOLE && nc + 16 * j >= at.n) continue;
      T* row = p + (int64_t)(nc + 16 * j) * ld + mc;
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        const int here = WHOLE ? 4 : at.m - mc - 16 * i;
        float v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          v[k] = (ADD && k < here ? to_f32(row[16 * i + k]) : 0.f) + acc[i][j][k];
        if (here >= 4) {
          store_vec<4>(row + 16 * i, v);
        } else {
#pragma unroll
          for (int k = 0; k < 3; ++k)
            if (k < here) put(row + 16 * i + k, v[k]);
        }
      }
    }
  }
  template <typename T, bool ADD, int TI, int TJ>
  static __device__ __forceinline__ void store_as(const MmOut& o, const MmPlace& at,
                                                  const f32x4_t (&acc)[TI][TJ]) {
    T* p = static_cast<T*>(o.p) + at.split * o.split_step;
    if (at.m0 + 16 * TI <= at.m && at.n0 + 16 * TJ <= at.n)
      store<T, true, ADD>(p, o.ld, at, acc);
    else
      store<T, false, ADD>(p, o.ld, at, acc);
  }
  template <int TI, int TJ>
  static __device__ __forceinline__ void run(const Args& e, const MmPlace& at,
                                             const f32x4_t (&acc)[TI][TJ]) {
    const MmOut& o = e.out[at.job];
    if (o.dtype == SM_BF16) store_as<bf16_t, false>(o, at, acc);
    else if (o.add) store_as<float, true>(o, at, acc);
    else store_as<float, false>(o, at, acc);
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

// The planes of a job's operands; a_plane and b_plane in bytes.
inline void set_planes(MmJob& j, int planes, int64_t a_plane, int64_t b_plane) {
  j.pairs = planes == 1 ? 1 : 6;
  j.parts = 1;
  j.a_plane = a_plane;
  j.b_plane = b_plane;
}

// Places in a workspace, each 256-byte aligned.
struct Places {
  char* base;
  size_t used = 0;
  template <typename T>
  T* take(int64_t n) {
    T* p = reinterpret_cast<T*>(base + used);
    used += ((size_t)n * sizeof(T) + 255) / 256 * 256;
    return p;
  }
};

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

// Launches the jobs of `a` (operands, extents, planes and splits are set).
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

#define SM_TRY(call)                                         \
  do {                                                       \
    if (hipError_t e_ = (call); e_ != hipSuccess) return e_; \
  } while (0)

}  // namespace sm
