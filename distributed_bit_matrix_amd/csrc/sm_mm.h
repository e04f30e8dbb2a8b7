// Matrix products of the feed-forward and loss operators on the matrix cores:
//   out[n][m] = sum over k of A(m, k) B(n, k),
// bfloat16 operands with float32 accumulators.  m counts features and n rows of
// activations: a lane's four accumulators of a 16x16 tile are four neighbouring
// features of one row, so what follows a product (a softmax over features, the
// gate's activation, a store) has them side by side.
//
// Operands lie as the caller has them: with k along the rows, or with k down the
// columns ("k-major": a weight whose rows are summed over, an activation whose
// rows are), read from LDS with transposing loads, so no transposed copy is
// ever made.  Slabs of 64 k go from memory to LDS through a buffer descriptor
// whose size ends at the matrix: rows past its end read as zeros, and no load
// is predicated.
//
// float32 operands are three bfloat16 planes each, whose sum is the value to 24
// bits; the product is the sum over the six pairs of planes that reach float32's
// precision ("segments" of one long k).  That runs at a sixth of the bfloat16
// rate, which is above what the float32 matrix instructions reach.
#pragma once

#include <algorithm>
#include <type_traits>

#include "sm_lds.h"

namespace sm {

constexpr int kSlab = 64;          // k of one slab
constexpr int kMaxSegs = 12;       // 6 pairs of planes, two products
constexpr int kMaxJobs = 3;

// One product of a launch.  Row lengths count elements.
struct MmJob {
  const char *a, *a2, *b;          // a2: the second weight of a paired product
  int64_t lda, ldb;
  int32_t m, n, k;
  int32_t segs, splits;            // splits: blocks that share a tile's k
  int32_t m_tiles, n_tiles;
  int32_t block0;                  // its first block
  int64_t a_seg[kMaxSegs], b_seg[kMaxSegs];   // bytes from a and b to a segment
};
// n_rows, k_rows: where not null, *n_rows replaces n of every job, *k_rows k.
struct MmArgs {
  MmJob job[kMaxJobs];
  int32_t jobs, blocks;
  const int32_t *n_rows, *k_rows;
};

// What an epilogue knows of its wave's part of a tile.
struct MmPlace {
  int job, split, m0, n0, m, n, lane;
};

template <int TM_, int TN_, int WM_, int WN_>
struct MmShape {
  static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = WN_;
  static constexpr int WAVES = WM * WN, TI = TM / WM / 16, TJ = TN / WN / 16;
  static constexpr int A_BYTES = TM * kSlab * 2, B_BYTES = TN * kSlab * 2;
  static constexpr int LDS = 2 * (A_BYTES + B_BYTES);
};

// One operand's slabs on their way to LDS.  Load q of a wave fills 1 KiB.
template <bool KM, int T, int Q>
struct MmSource {
  uint32_t off[Q];
  int chunk[Q];
  // row0: the tile's first row (k along rows) or column (k-major) is at base
  __device__ __forceinline__ void place(int wave, int lane, int64_t ld, int row_step) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int i = wave * Q + q;
      if constexpr (KM) {
        const int half = i >> 4, kr = 4 * (i & 15) + (lane >> 4), p = lane & 15;
        off[q] = (uint32_t)(kr * (ld * 2) + half * 256 + (((p >> 1) ^ km_swz(kr)) << 5) +
                            ((p & 1) << 4));
      } else {
        const int r = 8 * i + (lane >> 3), g = (lane & 7) ^ swz<128>(r);
        // paired: rows of 16 alternate between two matrices
        const int at = row_step == 2 ? (r >> 5) * 16 + (r & 15) : r;
        off[q] = (uint32_t)(at * (ld * 2) + g * 16);
        chunk[q] = g * 8;
      }
    }
  }
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t mm_rsrc(const char* p, int64_t bytes) {
  const int64_t cap = 0x7FFFFFFF;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p), 0,
                                           (int)(bytes < 0 ? 0 : bytes < cap ? bytes : cap),
                                           0x00020000);
}

// AKM, BKM: the operand is k-major.  PAIR: A's rows alternate in groups of 16
// between a and a2 (a tile has TM / 2 features of each).
template <bool AKM, bool BKM, bool PAIR, class Sh, class Epi>
__global__ __launch_bounds__(64 * Sh::WAVES, 2) void k_mm(MmArgs args, typename Epi::Args ea) {
  constexpr int TM = Sh::TM, TN = Sh::TN, TI = Sh::TI, TJ = Sh::TJ;
  constexpr int QA = Sh::A_BYTES / 1024 / Sh::WAVES, QB = Sh::B_BYTES / 1024 / Sh::WAVES;
  static_assert(!PAIR || (!AKM && QA == 4), "paired rows");
  __shared__ __align__(1024) char smem[Sh::LDS];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / Sh::WN, wn = wave % Sh::WN;

  int ji = 0;
#pragma unroll
  for (int i = 1; i < kMaxJobs; ++i)
    if (i < args.jobs && (int)blockIdx.x >= args.job[i].block0) ji = i;
  const MmJob& job = args.job[ji];
  const int n_all = args.n_rows ? *args.n_rows : job.n;
  const int k_all = args.k_rows ? *args.k_rows : job.k;
  const int m_tiles = job.m_tiles, n_tiles = args.n_rows ? (n_all + TN - 1) / TN : job.n_tiles;
  // Blocks go round the 8 XCDs: each gets a run of neighbouring tiles, in
  // groups of 4 tiles along n, so that its L2 holds what they share.
  const int total = m_tiles * n_tiles * job.splits;
  int at = blockIdx.x - job.block0;
  if (at >= total) return;
  {
    const int x = at & 7, q = total >> 3, r = total & 7;
    at = x * q + (x < r ? x : r) + (at >> 3);
  }
  const int split = at / (m_tiles * n_tiles);
  at -= split * m_tiles * n_tiles;
  const int group = at / (4 * m_tiles), g0 = group * 4;
  const int gn = n_tiles - g0 < 4 ? n_tiles - g0 : 4;
  at -= g0 * m_tiles;
  const int mt = at / gn, nt = g0 + at % gn;
  const int m0 = mt * (PAIR ? TM / 2 : TM), n0 = nt * TN;
  const int m_here = job.m - m0, n_here = n_all - n0 < TN ? n_all - n0 : TN;

  MmSource<AKM, TM, QA> sa;
  MmSource<BKM, TN, QB> sb;
  sa.place(wave, lane, job.lda, PAIR ? 2 : 1);
  sb.place(wave, lane, job.ldb, 1);
  const int64_t a0 = AKM ? (int64_t)m0 * 2 : (int64_t)m0 * job.lda * 2;
  const int64_t b0 = BKM ? (int64_t)n0 * 2 : (int64_t)n0 * job.ldb * 2;
  const int m_rows = PAIR ? (m_here < TM / 2 ? m_here : TM / 2) : (m_here < TM ? m_here : TM);
  const int per_seg = (k_all + kSlab - 1) / kSlab;
  const int slabs = per_seg * job.segs;
  const int per = (slabs + job.splits - 1) / job.splits;
  const int s0 = split * per, s1 = s0 + per < slabs ? s0 + per : slabs;

  auto issue = [&](int s, int stage) SM_INLINE {
    const int seg = s / per_seg, k0 = (s - seg * per_seg) * kSlab, left = k_all - k0;
    const int rows = left < kSlab ? left : kSlab;
    char* la = smem + stage * (Sh::A_BYTES + Sh::B_BYTES) + wave * QA * 1024;
    char* lb = smem + stage * (Sh::A_BYTES + Sh::B_BYTES) + Sh::A_BYTES + wave * QB * 1024;
    // bytes from the slab's base to the end of what may be read
    const int64_t a_at = a0 + job.a_seg[seg] + (AKM ? k0 * job.lda * 2 : (int64_t)k0 * 2);
    const int64_t b_at = b0 + job.b_seg[seg] + (BKM ? k0 * job.ldb * 2 : (int64_t)k0 * 2);
    const int64_t a_end = AKM ? ((rows - 1) * job.lda + ((m_here + 7) & ~7)) * 2
                              : ((m_rows - 1) * job.lda + ((left + 7) & ~7)) * 2;
    const int64_t b_end = BKM ? ((rows - 1) * job.ldb + ((n_all - n0 + 7) & ~7)) * 2
                              : ((n_here - 1) * job.ldb + ((left + 7) & ~7)) * 2;
    const auto ra = mm_rsrc(job.a + a_at, a_end);
    const auto ra2 = PAIR ? mm_rsrc(job.a2 + a_at, a_end) : ra;
    const auto rb = mm_rsrc(job.b + b_at, b_end);
#pragma unroll
    for (int q = 0; q < QA; ++q) {
      uint32_t o = sa.off[q];
      if constexpr (!AKM) o = sa.chunk[q] < left ? o : 0x80000000u;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(PAIR && q >= 2 ? ra2 : ra,
                                               (lds_void*)(la + q * 1024), 16, o, 0, 0, 0);
    }
#pragma unroll
    for (int q = 0; q < QB; ++q) {
      uint32_t o = sb.off[q];
      if constexpr (!BKM) o = sb.chunk[q] < left ? o : 0x80000000u;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(lb + q * 1024), 16, o, 0, 0, 0);
    }
  };

  // A fragment of MFMA tile t (16 rows from the wave's first) and k-step kk.
  // k along rows: one 16-byte read.  k-major: two transposing reads, 4 rows
  // apart, as in the layout's comment; the wave's columns begin at c0.
  constexpr int RA = TM / Sh::WM, RB = TN / Sh::WN;
  const int fa = AKM ? (wm * RA >> 7) * 16384 +
                           km_off<bf16_t>(8 * (lane >> 4) + ((lane & 15) >> 2),
                                          2 * (wm * RA & 127) + 8 * (lane & 3))
                     : lds_off<128>(wm * RA + (lane & 15), lane >> 4);
  const int fb = Sh::A_BYTES +
                 (BKM ? (wn * RB >> 7) * 16384 +
                            km_off<bf16_t>(8 * (lane >> 4) + ((lane & 15) >> 2),
                                           2 * (wn * RB & 127) + 8 * (lane & 3))
                      : lds_off<128>(wn * RB + (lane & 15), lane >> 4));
  auto frag = [&](auto km, const char* st, int base, int t, int kk) SM_INLINE -> bf16x8_t {
    if constexpr (decltype(km)::value) {
      const char* p = st + (base ^ (t << 5)) + kk * 8192;
      const u32x2_t lo = lds_read_tr16(p), hi = lds_read_tr16(p + 1024);
      return __builtin_bit_cast(bf16x8_t, u32x4_t{lo[0], lo[1], hi[0], hi[1]});
    } else {
      return *reinterpret_cast<const bf16x8_t*>(st + (base ^ (kk << 6)) + t * 2048);
    }
  };

  f32x4_t acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  if (s0 < s1) issue(s0, 0);
  for (int s = s0; s < s1; ++s) {
    const int stage = (s - s0) & 1;
    wait_vmcnt<0>();
    wait_lgkmcnt0();
    __builtin_amdgcn_s_barrier();
    if (s + 1 < s1) issue(s + 1, stage ^ 1);
    const char* st = smem + stage * (Sh::A_BYTES + Sh::B_BYTES);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      bf16x8_t a[TI], b[TJ];
#pragma unroll
      for (int j = 0; j < TJ; ++j) b[j] = frag(std::bool_constant<BKM>{}, st, fb, j, kk);
#pragma unroll
      for (int i = 0; i < TI; ++i) a[i] = frag(std::bool_constant<AKM>{}, st, fa, i, kk);
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
    }
  }
  const MmPlace at_wave{ji, split, m0 + wm * (PAIR ? RA / 2 : RA), n0 + wn * RB, job.m, n_all, lane};
  Epi::template run<TI, TJ>(ea, at_wave, acc);
}

}  // namespace sm
