// Epilogues, operand copies and launches shared by the feed-forward and loss
// operators.
#pragma once

#include "sm_mm.h"
#include "sm_rows.h"

namespace sm {

// 16 rows of an epilogue's F features on their way to memory.  In the accumulators
// a lane has 4 features of one row: stores from there write 32 bytes of each of 16
// rows (8 us for a tile of 256 x 256 bfloat16, as long as 5 slabs).  Through LDS
// they become 16 bytes a lane of whole lines.  Rows are swizzled by 16-byte pieces:
// lanes of 16 rows write, and lanes of one row read, distinct banks.  A wave uses
// its own LDS, two buffers (three of bfloat16) in turn.
template <typename T, int F>
struct MmRows {
  static constexpr int ES = (int)sizeof(T), RB = F * ES, CR = RB / 16, V = 16 / ES;
  static_assert(CR >= 4 && CR <= 32 && (ES == 4 ? 2 : 3) * 16 * RB <= 16384, "rows of an epilogue");
  char* lds;
  int lane;
  __device__ __forceinline__ char* piece(int buf, int row, int chunk) const {
    return lds + buf * 16 * RB + row * RB + ((chunk ^ (row & (CR - 1))) << 4);
  }
  // features 16 i + 4 (lane / 16) .. +3 of row lane % 16
  __device__ __forceinline__ void put(int buf, int i, const f32x4_t& v) const {
    const int row = lane & 15, g = 4 * i + (lane >> 4);      // group of 4 features
    if constexpr (ES == 4)
      *reinterpret_cast<f32x4_t*>(piece(buf, row, g)) = v;
    else
      *reinterpret_cast<u32x2_t*>(piece(buf, row, g >> 1) + (g & 1) * 8) =
          u32x2_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
  }
  // the first `rows` of the 16 and `cols` of the F to p; ADD: to what is there
  template <bool ADD = false>
  __device__ __forceinline__ void flush(int buf, T* p, int64_t ld, int rows, int cols) const {
#pragma unroll
    for (int it = 0; it < CR / 4; ++it) {
      const int row = it * (64 / CR) + lane / CR, chunk = lane % CR, c = chunk * V;
      const u32x4_t t = *reinterpret_cast<const u32x4_t*>(piece(buf, row, chunk));
      if (row >= rows || c >= cols) continue;
      T* q = p + row * ld + c;
      if constexpr (ES == 4) {
        float v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = __uint_as_float(t[k]);
        if (c + V <= cols) {
          if constexpr (ADD) {
            const u32x4_a4 old = *reinterpret_cast<const u32x4_a4*>(q);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] += __uint_as_float(old[k]);
          }
          store_vec<4>(q, v);
        } else {
#pragma unroll
          for (int k = 0; k < 3; ++k)
            if (c + k < cols) q[k] = (ADD ? q[k] : 0.f) + v[k];
        }
      } else {
        if (c + V <= cols) {
          *reinterpret_cast<u32x4_a2*>(q) = u32x4_a2{t[0], t[1], t[2], t[3]};
        } else {
#pragma unroll
          for (int k = 0; k < 7; ++k)
            if (c + k < cols) q[k] = (bf16_t)(t[k / 2] >> (16 * (k & 1)));
        }
      }
    }
  }
};

// 16 rows of F features to P planes, `plane` entries apart, from accumulators
// v[i] as `put` takes them.
template <int P, int F>
__device__ __forceinline__ void put_planes(const MmPlace& at, const f32x4_t (&v)[F / 16], bf16_t* p,
                                           int64_t plane, int64_t ld, int rows, int cols) {
  const MmRows<bf16_t, F> out{at.lds, at.lane};
  if constexpr (P == 1) {
#pragma unroll
    for (int i = 0; i < F / 16; ++i) out.put(0, i, v[i]);
    out.flush(0, p, ld, rows, cols);
  } else {
    f32x4_t left[F / 16];
#pragma unroll
    for (int i = 0; i < F / 16; ++i) left[i] = v[i];
#pragma unroll
    for (int q = 0; q < P; ++q) {
#pragma unroll
      for (int i = 0; i < F / 16; ++i) {
        f32x4_t part = left[i];
        if (q == 0)
#pragma unroll
          for (int k = 0; k < 4; ++k) part[k] = first_plane(part[k]);
        out.put(q & 1, i, part);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float hi = bf16_to_f32(f32_to_bf16(part[k]));
          left[i][k] = __builtin_isfinite(hi) ? left[i][k] - hi : 0.f;
        }
      }
      out.flush(q & 1, p + q * plane, ld, rows, cols);
    }
  }
}

// Four neighbouring values to P planes, `plane` entries apart; 8-byte aligned.  Each
// plane has what the ones before it leave, rounded: three hold float32's 24 bits.  A
// value that is not finite is in the first.
template <int P>
__device__ __forceinline__ void store_mid(bf16_t* p, int64_t plane, f32x4_t v) {
#pragma unroll
  for (int q = 0; q < P; ++q) {
    f32x4_t part = v;
    if (P > 1 && q == 0)
#pragma unroll
      for (int k = 0; k < 4; ++k) part[k] = first_plane(part[k]);
    const uint32_t lo = pack_bf16(part[0], part[1]), hi = pack_bf16(part[2], part[3]);
    *reinterpret_cast<u32x2_t*>(p + q * plane) = u32x2_t{lo, hi};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float t = bf16_to_f32((bf16_t)((k < 2 ? lo : hi) >> (16 * (k & 1))));
      v[k] = __builtin_isfinite(t) ? v[k] - t : 0.f;
    }
  }
}

// The product itself: to an array of a caller's type, or (parts) to float32
// sums of a split, which a later launch joins.
struct MmOut {
  void* p;
  int64_t ld;
  int64_t split_step;      // elements from one split's sums to the next
  int32_t dtype, add;      // add: to what is there (float32)
  const float* by;         // a factor, or null
};
struct EpiStore {
  struct Args {
    MmOut out[kMaxJobs];
  };
  template <typename T, bool ADD, int TI, int TJ>
  static __device__ __forceinline__ void store(const MmOut& o, const MmPlace& at,
                                               const f32x4_t (&acc)[TI][TJ]) {
    const MmRows<T, 16 * TI> rows{at.lds, at.lane};
    T* p = static_cast<T*>(o.p) + at.split * o.split_step + at.m0;
    const float by = o.by ? *o.by : 1.f;
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
#pragma unroll
      for (int i = 0; i < TI; ++i) rows.put(j & 1, i, acc[i][j] * by);
      const int n = at.n0 + 16 * j;
      rows.template flush<ADD>(j & 1, p + (int64_t)n * o.ld, o.ld, at.n - n, at.m - at.m0);
    }
  }
  template <int TI, int TJ>
  static __device__ __forceinline__ void run(const Args& e, const MmPlace& at,
                                             const f32x4_t (&acc)[TI][TJ]) {
    const MmOut& o = e.out[at.job];
    if (o.dtype == SM_BF16) store<bf16_t, false>(o, at, acc);
    else if (o.add) store<float, true>(o, at, acc);
    else store<float, false>(o, at, acc);
  }
};

// Rows of a caller's matrix as `planes` bfloat16 planes of row length ld, its
// pad zero.  list, count: rows list[0 .. *count), or all where list is null.
struct PlanesArgs {
  const void* src;
  int64_t stride;
  int64_t rows;
  int32_t cols, ld;
  const int32_t *list, *count;
  bf16_t* dst;
};
// Copies of one dtype and number of planes, in one launch.
constexpr int kMaxPlanes = 5;
struct PlanesJobs {
  PlanesArgs job[kMaxPlanes];
  int32_t jobs;
  int32_t block0[kMaxPlanes];
};
hipError_t launch_planes(PlanesJobs& a, int32_t dtype, hipStream_t s);

// Sums of splits joined: out[r][c] = by * sum over s of part[s][at(r)][c] (plus
// what is there), at(r) = pos[r], or r where pos is null; a row whose pos is
// negative is zero.
struct JoinArgs {
  const float* part;
  int64_t split_step, part_ld;
  int32_t splits;
  const int32_t* pos;
  int64_t rows;
  int32_t cols, dtype, add;
  void* out;
  int64_t ld;
  const float* by;         // a factor, or null
};
struct JoinJobs {
  JoinArgs job[kMaxJobs];
  int32_t jobs;
  int32_t block0[kMaxJobs];
};
hipError_t launch_join(JoinJobs& a, hipStream_t s);      // in one launch

// The row length of an operand copy: whole pieces of 128 bytes, an odd number of
// them.  Rows a power of two apart meet in the same memory channels: 8192^3 with
// both operands k along rows of 16 KiB 1122 TFLOP/s, with rows 128 bytes longer
// 1322.
inline int64_t operand_ld(int64_t cols) { return ((cols + 63) / 64 | 1) * 64; }

hipError_t launch_zero(void* p, int32_t dtype, int64_t n, hipStream_t s);

// Whether a matrix can be an operand where it lies: rows of whole 16-byte
// pieces, and offsets within a tile of 31 bits.
inline bool operand_fits(const void* p, int32_t dtype, int64_t cols, int64_t stride) {
  return dtype == SM_BF16 && (uintptr_t)p % 16 == 0 && cols % 8 == 0 && stride % 8 == 0 &&
         stride <= ((int64_t)1 << 21);
}

// The planes of a job's operands, (1, 1), (1, 2), (2, 1) or (3, 3); a_plane and
// b_plane in bytes.
inline void set_planes(MmJob& j, int a_planes, int b_planes, int64_t a_plane, int64_t b_plane) {
  j.pairs = a_planes * b_planes == 9 ? 6 : a_planes * b_planes;
  j.code = a_planes * b_planes == 9 ? kPairCode
           : b_planes == 2          ? kPairOneTwo
           : a_planes == 2          ? kPairTwoOne
                                    : 0;
  j.parts = 1;
  j.a_plane = a_plane;
  j.b_plane = b_plane;
}

// A product's sums of splits, for a launch of its own that joins them.
inline MmOut sums_out(float* sums, int64_t m, int64_t n) {
  const int64_t ld = round_up(m, 4);
  return {sums, ld, n * ld, SM_F32, 0, nullptr};
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

// A product that is to be launched: its extents, in slabs of k; whether its k may
// be split.
struct MmSize {
  int64_t m, n, slabs;
  bool may_split;
};
// Tiles of 256 x 256 or 128 x 128, and how many blocks share a tile's k.
struct MmPlan {
  bool wide;
  int splits[kMaxJobs];
};
// The plan whose blocks, dealt out longest first to the CUs as they fall free, are
// done first.  A slab takes 1.65 us in a wide tile and 1.0 in one of two narrow
// ones on a CU; a block 5 us more for its first loads and its epilogue; a split's
// sums go to memory and back.  That is of products with k along rows and short
// epilogues.  Others take longer than planned: the block's gradient of 12288 rows of 768 x
// 2048, bfloat16, 163 us for 50 in its first launch, whose epilogue moves 0.9 MB a block,
// and 270 for 207 in its second, with operands k-major.
MmPlan plan_products(const MmSize* sizes, int jobs);

template <bool AKM, bool BKM, bool PAIR, class Sh, class Epi>
hipError_t run_mm_as(MmArgs& a, const typename Epi::Args& e, bool both, hipStream_t s) {
  int64_t blocks = 0;
  for (int i = 0; i < a.jobs; ++i) {
    MmJob& j = a.job[i];
    const int tm = PAIR ? Sh::TM / 2 : Sh::TM;
    j.m_tiles = (j.m + tm - 1) / tm;
    j.n_tiles = (j.n + Sh::TN - 1) / Sh::TN;
    j.block0 = (int)blocks;
    blocks += (int64_t)j.m_tiles * j.n_tiles * j.splits;
    if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  }
  if (blocks == 0) return hipSuccess;
  const dim3 grid((unsigned)blocks), block(64 * Sh::WAVES);
  if constexpr (AKM && !PAIR && std::is_same_v<Epi, EpiStore>) {
    if (both) {
      hipLaunchKernelGGL((k_mm_both<Sh, Epi>), grid, block, 0, s, a, e);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((k_mm<AKM, BKM, PAIR, Sh, Epi>), grid, block, 0, s, a, e);
  return hipGetLastError();
}
// Launches the jobs of `a` (operands, extents, planes and splits are set).
template <bool AKM, bool BKM, bool PAIR, class Epi>
hipError_t run_mm(MmArgs& a, const typename Epi::Args& e, bool wide, hipStream_t s) {
  return wide ? run_mm_as<AKM, BKM, PAIR, MmShape<256, 256, 2, 4>, Epi>(a, e, false, s)
              : run_mm_as<AKM, BKM, PAIR, MmShape<128, 128, 2, 2>, Epi>(a, e, false, s);
}

// Products with a k-major A that end in arrays (or in sums of splits, joined here),
// all in one launch.
struct MmStores {
  MmArgs a{};
  EpiStore::Args e{};
  JoinJobs join{};
  // job j, whose rows, times *by, go to dst; sums: where those of its splits go, if
  // it has any
  void add(const MmJob& j, bool b_km, void* dst, int32_t dtype, int32_t accumulate, float* sums,
           int splits, const float* by = nullptr);
  hipError_t run(bool wide, hipStream_t s);
  hipError_t joins(hipStream_t s);
};

#define SM_TRY(call)                                         \
  do {                                                       \
    if (hipError_t e_ = (call); e_ != hipSuccess) return e_; \
  } while (0)

}  // namespace sm
