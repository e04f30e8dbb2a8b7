// Device helpers shared by the row operators (layer norm, embedding): pieces of
// rows at any element alignment, and sums within lane groups.
#pragma once

#include "sm_internal.h"

namespace sm {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16_t v) { return bf16_to_f32(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(bf16_t* p, float v) { *p = f32_to_bf16(v); }

// A row of odd length starts at an address that is a multiple of its element
// size only.  Global memory instructions of 16 bytes take such addresses, so
// the vector types below carry the element's alignment and rows of every
// length move in 16-byte pieces.
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_a4 __attribute__((ext_vector_type(2), aligned(4)));
typedef uint32_t u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

// A pass that moves more than this reads its input with the non-temporal hint:
// the last-level cache (256 MB) cannot hold it for the next pass, and without
// the hint it writes its dirty lines back while this pass reads.  Measured:
// layer norm of 65536 x 1024 float32 90 -> 79 us, backward 147 -> 123 us, the
// embedding sums of 65536 x 2048 122 -> 91 us; at 100 and 150 MB the hint
// costs 10% (32768 x 768 bfloat16 17.7 -> 19.8 us, backward 27.9 -> 30.4 us).
constexpr int64_t kCacheBytes = (int64_t)256 << 20;

// V consecutive entries as they lie in memory (V = 1, or 8 bytes or a multiple
// of 16).  Loading and widening are apart, so that a kernel can have all its
// loads under way before the first value is looked at.
template <typename T, int V>
struct Piece {
  static constexpr int kWords = V * (int)sizeof(T) / 4;
  uint32_t w[kWords];
  template <bool NT = false>
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kWords == 2) {
      const u32x2_a2* q = reinterpret_cast<const u32x2_a2*>(p);
      const u32x2_a2 t = NT ? __builtin_nontemporal_load(q) : *q;
      w[0] = t[0];
      w[1] = t[1];
    } else {
#pragma unroll
      for (int k = 0; k < kWords; k += 4) {
        uint32_t t[4];
        if constexpr (sizeof(T) == 4) {
          const u32x4_a4* q = reinterpret_cast<const u32x4_a4*>(p + k);
          const u32x4_a4 v = NT ? __builtin_nontemporal_load(q) : *q;
          t[0] = v[0], t[1] = v[1], t[2] = v[2], t[3] = v[3];
        } else {
          const u32x4_a2* q = reinterpret_cast<const u32x4_a2*>(p + 2 * k);
          const u32x4_a2 v = NT ? __builtin_nontemporal_load(q) : *q;
          t[0] = v[0], t[1] = v[1], t[2] = v[2], t[3] = v[3];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) w[k + j] = t[j];
      }
    }
  }
  __device__ __forceinline__ float operator[](int k) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[k]);
    else return __uint_as_float(k & 1 ? w[k >> 1] & 0xFFFF0000u : w[k >> 1] << 16);
  }
};
template <typename T>
struct Piece<T, 1> {
  T v;
  template <bool NT = false>
  __device__ __forceinline__ void load(const T* p) {
    v = *p;
  }
  __device__ __forceinline__ float operator[](int) const { return to_f32(v); }
};

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return (uint32_t)f32_to_bf16(a) | ((uint32_t)f32_to_bf16(b) << 16);
}
// What the first of several bfloat16 planes of v is rounded from.  A finite v past the
// largest bfloat16 has that one, and the later planes what is left: nearest rounding
// would make it an infinity.
__device__ __forceinline__ float first_plane(float v) {
  constexpr float kMost = 0x1.FEp127f;
  return __builtin_isfinite(v) ? __builtin_amdgcn_fmed3f(v, -kMost, kMost) : v;
}
template <int V>
__device__ __forceinline__ void store_vec(float* p, const float (&v)[V]) {
  if constexpr (V == 1) {
    *p = v[0];
  } else {
#pragma unroll
    for (int k = 0; k < V; k += 4)
      *reinterpret_cast<u32x4_a4*>(p + k) =
          u32x4_a4{__float_as_uint(v[k]), __float_as_uint(v[k + 1]), __float_as_uint(v[k + 2]),
                   __float_as_uint(v[k + 3])};
  }
}
template <int V>
__device__ __forceinline__ void store_vec(bf16_t* p, const float (&v)[V]) {
  if constexpr (V == 1) {
    *p = f32_to_bf16(v[0]);
  } else if constexpr (V == 4) {
    *reinterpret_cast<u32x2_a2*>(p) = u32x2_a2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
  } else {
#pragma unroll
    for (int k = 0; k < V; k += 8)
      *reinterpret_cast<u32x4_a2*>(p + k) =
          u32x4_a2{pack_bf16(v[k], v[k + 1]), pack_bf16(v[k + 2], v[k + 3]),
                   pack_bf16(v[k + 4], v[k + 5]), pack_bf16(v[k + 6], v[k + 7])};
  }
}

// Where a lane's piece of a row of `cols` >= V entries lies if it would begin
// at c: a piece that would pass the row's end begins earlier, and its first
// `skip` entries belong to the lane before it (all V: the piece has none).
// So every lane loads a whole piece inside the row.
template <int V>
struct Place {
  int c, skip;
  __device__ __forceinline__ Place(int at, int cols) {
    const int over = at + V - cols;
    skip = over <= 0 ? 0 : over < V ? over : V;
    c = over <= 0 ? at : cols - V;
  }
};
// The entries of v that are the lane's own, to p.
template <int V, typename T>
__device__ __forceinline__ void store_own(T* p, int skip, const float (&v)[V]) {
  if (skip == 0) {
    store_vec<V>(p, v);
  } else if (skip < V) {
#pragma unroll
    for (int k = 1; k < V; ++k)
      if (k >= skip) put(p + k, v[k]);
  }
}

// Sum over aligned groups of W lanes (W a power of two, at most 64), in a
// fixed order; the result reaches every lane of the group.  Up to 16 lanes meet
// by data-parallel moves within a row of 16 (a shuffle would take a round trip
// to LDS); four rows of 16 meet through scalars.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF,
                                                        false));
}
template <int W>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (W >= 2) v = dpp_add<0xB1>(v);     // quad_perm 1,0,3,2
  if constexpr (W >= 4) v = dpp_add<0x4E>(v);     // quad_perm 2,3,0,1
  if constexpr (W >= 8) v = dpp_add<0x141>(v);    // row_half_mirror
  if constexpr (W >= 16) v = dpp_add<0x140>(v);   // row_mirror
  if constexpr (W == 32) v += __shfl_xor(v, 16);
  if constexpr (W == 64) {
    const int i = __float_as_int(v);
    v = (__int_as_float(__builtin_amdgcn_readlane(i, 0)) +
         __int_as_float(__builtin_amdgcn_readlane(i, 16))) +
        (__int_as_float(__builtin_amdgcn_readlane(i, 32)) +
         __int_as_float(__builtin_amdgcn_readlane(i, 48)));
  }
  return v;
}

}  // namespace sm
