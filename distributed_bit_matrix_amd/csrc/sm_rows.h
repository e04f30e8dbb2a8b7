// Device helpers shared by the row operators (layer norm, embedding): wide
// loads and stores at any element alignment, and sums within lane groups.
#pragma once

#include "sm_internal.h"

namespace sm {

// A row of odd length starts at an address that is a multiple of its element
// size only.  Global memory instructions of 16 bytes take such addresses, so
// the vector types below carry the element's alignment and rows of every
// length move in 16-byte pieces.
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));
typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16_t v) { return bf16_to_f32(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(bf16_t* p, float v) { *p = f32_to_bf16(v); }

template <int V>
__device__ __forceinline__ void load_vec(const float* p, float (&v)[V]) {
  static_assert(V % 4 == 0, "pieces of 4");
#pragma unroll
  for (int k = 0; k < V; k += 4) {
    f32x4_a4 t = *reinterpret_cast<const f32x4_a4*>(p + k);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[k + j] = t[j];
  }
}
template <int V>
__device__ __forceinline__ void load_vec(const bf16_t* p, float (&v)[V]) {
  static_assert(V == 4 || V % 8 == 0, "pieces of 4 or 8");
  if constexpr (V == 4) {
    u32x2_a2 t = *reinterpret_cast<const u32x2_a2*>(p);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      v[2 * j] = __uint_as_float(t[j] << 16);
      v[2 * j + 1] = __uint_as_float(t[j] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int k = 0; k < V; k += 8) {
      u32x4_a2 t = *reinterpret_cast<const u32x4_a2*>(p + k);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[k + 2 * j] = __uint_as_float(t[j] << 16);
        v[k + 2 * j + 1] = __uint_as_float(t[j] & 0xFFFF0000u);
      }
    }
  }
}
template <int V>
__device__ __forceinline__ void store_vec(float* p, const float (&v)[V]) {
#pragma unroll
  for (int k = 0; k < V; k += 4)
    *reinterpret_cast<f32x4_a4*>(p + k) = f32x4_a4{v[k], v[k + 1], v[k + 2], v[k + 3]};
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return (uint32_t)f32_to_bf16(a) | ((uint32_t)f32_to_bf16(b) << 16);
}
template <int V>
__device__ __forceinline__ void store_vec(bf16_t* p, const float (&v)[V]) {
  if constexpr (V == 4) {
    *reinterpret_cast<u32x2_a2*>(p) = u32x2_a2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
  } else {
#pragma unroll
    for (int k = 0; k < V; k += 8)
      *reinterpret_cast<u32x4_a2*>(p + k) =
          u32x4_a2{pack_bf16(v[k], v[k + 1]), pack_bf16(v[k + 2], v[k + 3]),
                   pack_bf16(v[k + 4], v[k + 5]), pack_bf16(v[k + 6], v[k + 7])};
  }
}
// The first `have` of V elements (all, when have >= V); the rest read as 0.
template <int V, typename T>
__device__ __forceinline__ void load_part(const T* p, int have, float (&v)[V]) {
  if (have >= V) {
    load_vec<V>(p, v);
    return;
  }
#pragma unroll
  for (int k = 0; k < V; ++k) v[k] = k < have ? to_f32(p[k]) : 0.f;
}
template <int V, typename T>
__device__ __forceinline__ void store_part(T* p, int have, const float (&v)[V]) {
  if (have >= V) {
    store_vec<V>(p, v);
    return;
  }
#pragma unroll
  for (int k = 0; k < V; ++k)
    if (k < have) put(p + k, v[k]);
}

// Sum over aligned groups of W lanes (W a power of two, at most 64), in a
// fixed order; the result reaches every lane of the group.
template <int W>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

}  // namespace sm
