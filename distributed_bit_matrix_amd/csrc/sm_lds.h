// LDS layouts, transposing reads and counter waits of the matrix-core kernels.
#pragma once

#include "sm_internal.h"

namespace sm {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void lds_void;
// the kernel's helper lambdas take register arrays by reference: they must
// be inlined, or the arrays would live in scratch memory
#define SM_INLINE __attribute__((always_inline))

// LDS image of one k-slab of an operand tile: RB bytes per row (64 or 128),
// 16-byte chunks XOR-swizzled by row.  A fragment read is a ds_read_b128
// with 16 lanes on 16 consecutive rows and lane groups 16 apart on
// neighbouring chunks.  The LDS serves such a read per half-wave: it is
// free of bank conflicts when the 32 lanes of each half hit 32 distinct
// 16-byte units modulo 512 bytes (measured on gfx950 with the
// SQ_LDS_BANK_CONFLICT counter over several lane patterns; a swizzle that
// only separates groups of 8 or 16 lanes left a 2-way conflict).  Rows 4
// apart (128-byte rows) or 8 apart (64-byte rows) share a unit modulo 512
// bytes, so the swizzle separates exactly those.  It depends on row bits
// 0..3 only, so rows 16 apart share it and a fragment offset steps by a
// constant 16*RB bytes per 16-row tile.
template <int RB>
__host__ __device__ constexpr int swz(int row) {
  if constexpr (RB == 128) return (row >> 1) & 7;
  else return (((row >> 3) & 1) << 1) | ((row >> 2) & 1);
}
template <int RB>
__host__ __device__ constexpr int lds_off(int row, int chunk) {
  return row * RB + ((chunk ^ swz<RB>(row)) << 4);
}
// Compile-time checks of the layout: constant 16-row stride, a bijection of
// each row's chunks, and distinct 16-byte units modulo 512 bytes in each
// half-wave of a fragment read (lane l: row l % 16, chunk 4 kk + l / 16).
template <int RB>
constexpr bool slab_layout_ok() {
  constexpr int CPR = RB / 16;
  for (int r0 = 0; r0 < 256; r0 += 16) {
    for (int ch = 0; ch < CPR; ++ch)
      for (int r = 0; r < 16; ++r)
        if (lds_off<RB>(r0 + r, ch) != lds_off<RB>(r, ch) + r0 * RB) return false;
    for (int r = 0; r < 16; ++r) {
      unsigned seen = 0;
      for (int ch = 0; ch < CPR; ++ch) seen |= 1u << ((lds_off<RB>(r, ch) - r * RB) / 16);
      if (seen != (1u << CPR) - 1) return false;
    }
    for (int kk = 0; kk < CPR / 4; ++kk)
      for (int half = 0; half < 2; ++half) {
        unsigned seen = 0;
        for (int l = 32 * half; l < 32 * half + 32; ++l) {
          const int unit = (lds_off<RB>(r0 + (l & 15), 4 * kk + (l >> 4)) % 512) / 16;
          if (seen & (1u << unit)) return false;
          seen |= 1u << unit;
        }
      }
  }
  return true;
}
static_assert(slab_layout_ok<64>() && slab_layout_ok<128>(), "LDS slab swizzle");

// k-major operand tiles (an X block with k down its columns): LDS row = k
// within the slab, W * sizeof(T) bytes per row (the W output rows or columns
// of the tile), 32-byte chunks XOR-swizzled by row bits 0, 1 and 3.
// The 16 lanes of a transposing fragment read cover 4 consecutive rows of
// one chunk, and lane groups 16 apart read rows 8 apart; both then land in
// distinct bank groups.  The swizzle ignores row bit 2, so the second read
// of a fragment (4 rows down) is a constant offset away.
__host__ __device__ constexpr int km_swz(int row) { return (row & 3) ^ (((row >> 3) & 1) << 2); }
template <typename T, int W = 128>
__host__ __device__ constexpr int km_off(int row, int byte) {
  return row * (W * (int)sizeof(T)) + ((((byte >> 5) ^ km_swz(row)) << 5) | (byte & 31));
}
// Checks: a bijection of each row's chunks, and for the transposing read
// (lane j of a 16-lane group at row r0 + j/4, byte c*32 + 8*(j%4)) 16
// distinct 8-byte slots in 128 bytes, with lane groups 8 rows apart in the
// other half of 256 bytes.
constexpr bool km_layout_ok() {
  for (int r0 = 0; r0 < 64; r0 += 4)
    for (int c = 0; c < 8; ++c) {
      unsigned seen = 0, seen2 = 0;
      for (int j = 0; j < 16; ++j) {
        const int o = km_off<bf16_t>(r0 + j / 4, c * 32 + 8 * (j % 4));
        const int slot = (o % 128) / 8;
        if (seen & (1u << slot)) return false;
        seen |= 1u << slot;
        if (km_off<bf16_t>(r0 + 4 + j / 4, c * 32 + 8 * (j % 4)) != o + 4 * 256) {
          if ((r0 & 4) == 0) return false;
        }
        const int o8 = km_off<bf16_t>((r0 ^ 8) + j / 4, c * 32 + 8 * (j % 4));
        if ((o8 % 256) / 128 == (o % 256) / 128) return false;
        seen2 |= 1u << ((o8 % 128) / 8);
      }
      if (seen2 != 0xFFFFu) return false;
    }
  return true;
}
static_assert(km_layout_ok(), "k-major LDS swizzle");

typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4_t lds_i16x4;
// Transposing LDS read (ds_read_b64_tr_b16): within each group of 16 lanes,
// lane i receives element i % 4 of the 8 bytes addressed by lane
// 4 e + i / 4, for e = 0..3 (16-bit elements).
__device__ __forceinline__ u32x2_t lds_read_tr16(const char* p) {
  i16x4_t v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (lds_i16x4*)(__attribute__((address_space(3))) char*)p);
  return __builtin_bit_cast(u32x2_t, v);
}

// A uniform pointer made opaque to the optimizer (an empty asm statement
// that keeps it in scalar registers), so that it cannot be folded with
// per-lane offsets into 64-bit vector addresses carried across the loop: a
// load then keeps the scalar-base + 32-bit vector-offset form.
__device__ __forceinline__ const char* scalar_ptr(const char* p) {
  uint64_t v = reinterpret_cast<uint64_t>(p);
  asm volatile("" : "+s"(v));
  return reinterpret_cast<const char*>(v);
}

// s_waitcnt with only the vector-memory counter constrained (gfx9 encoding:
// vmcnt in bits 3:0 and 15:14, expcnt 6:4, lgkmcnt 11:8).
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | (((N >> 4) & 3) << 14));
}

// s_waitcnt lgkmcnt(0): this wave's LDS reads (and scalar loads) have
// returned; the vector-memory and export counters are left alone.
__device__ __forceinline__ void wait_lgkmcnt0() {
  __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (3 << 14));
}

}  // namespace sm
