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
//
// Bound by the chip's power: 4096 x 4096 x 16384 463 us (1190 TFLOP/s); 16384 x 8192 x
// 768 of uniform values 193 us, of zeros 144.
#pragma once

#include <algorithm>
#include <type_traits>

#include "sm_lds.h"

namespace sm {

constexpr int kSlab = 64;          // k of one slab
constexpr int kMaxJobs = 4;

// The pairs of planes of a float32 product: those whose products reach 2^-24 of
// the largest, the small ones first: (2,0) (1,1) (0,2) (1,0) (0,1) (0,0), as
// codes a + 4 b in four bits each.  Products of one plane with two: (0,1) (0,0),
// or (1,0) (0,0).
constexpr int kPairCode = 2 | (1 + 4) << 4 | (2 * 4) << 8 | 1 << 12 | 4 << 16;
constexpr int kPairOneTwo = 4, kPairTwoOne = 1;

// One product of a launch.  Row lengths count elements.
struct MmJob {
  const char *a, *a2, *b;          // a2: the second weight of a paired product
  const int32_t *n_rows, *k_rows;  // where not null, *n_rows replaces n, *k_rows k
  int64_t lda, ldb;
  int32_t m, n, k;
  int32_t pairs, code, parts;      // of planes, 1, 2 or 6; products that are summed: 1 or 2
  int32_t splits;                  // blocks that share a tile's k
  int32_t m_tiles, n_tiles;
  int32_t block0;                  // its first block
  int32_t b_km;                    // whether b is k-major, in launches of both kinds
  int64_t a_plane, b_plane;        // bytes from one plane to the next
  int64_t a_part, b_part;          // bytes to the second product's operands
};
struct MmArgs {
  MmJob job[kMaxJobs];
  int32_t jobs;
};

// What an epilogue knows of its wave's part of a tile; lds: 16 KiB of its own.
struct MmPlace {
  int job, split, m0, n0, m, n, lane;
  char* lds;
};

template <int TM_, int TN_, int WM_, int WN_, int WPE_ = 2>
struct MmShape {
  static constexpr int WPE = WPE_;
  static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = WN_;
  static constexpr int WAVES = WM * WN, TI = TM / WM / 16, TJ = TN / WN / 16;
  static constexpr int A_BYTES = TM * kSlab * 2, B_BYTES = TN * kSlab * 2;
  static constexpr int LDS = 2 * (A_BYTES + B_BYTES);
  static_assert(LDS / WAVES >= 16384, "an epilogue's LDS");
};

// Where a lane's 16 bytes of load q of a slab lie: load q of a wave fills the
// 1 KiB of LDS after the one before it, the layouts' swizzles are applied by the
// choice of global bytes.  k along rows: 8 rows of a load, whose swizzles repeat
// every two loads; k-major: 4 rows (of 128 columns each), every four.  So two
// offsets serve all loads, the rest is uniform.
template <bool KM, bool PAIR>
struct MmSource {
  uint32_t off[2];
  int chunk;                // k along rows: first k of the lane's bytes (load 0; load 1: ^ 32)
  int64_t row_bytes;
  __device__ __forceinline__ void place(int lane, int64_t ld) {
    row_bytes = ld * 2;
    if constexpr (KM) {
      const int p = lane & 15, kr = lane >> 4;
#pragma unroll
      for (int v = 0; v < 2; ++v)
        off[v] = (uint32_t)(kr * row_bytes +
                            ((((p >> 1) ^ km_swz(kr + 8 * v)) << 5) | (p & 1) << 4));
    } else {
      const int r = lane >> 3, g = (lane & 7) ^ swz<128>(r);
      chunk = g * 8;
      off[0] = (uint32_t)(r * row_bytes + g * 16);
      off[1] = (uint32_t)((r + 8) * row_bytes + (g ^ 4) * 16);
    }
  }
  // The offsets of a slab with `left` k to the end: what is past it is out of
  // any descriptor's range.
  __device__ __forceinline__ void slab(int left, uint32_t (&o)[2]) const {
    o[0] = KM || chunk < left ? off[0] : 0x80000000u;
    o[1] = KM || (chunk ^ 32) < left ? off[1] : 0x80000000u;
    // (opaque, or the loads' sums would be held in registers of their own)
    if constexpr (KM) asm volatile("" : "+v"(o[0]), "+v"(o[1]));
  }
  // load i of the operand's tile
  __device__ __forceinline__ uint32_t at(const uint32_t (&o)[2], int i) const {
    if constexpr (KM)
      return o[(i >> 1) & 1] + (uint32_t)(4 * (i & 15) * row_bytes + (i >> 4) * 256);
    // 16 rows of a group; paired, groups alternate between two matrices
    return o[i & 1] + (uint32_t)((PAIR ? i >> 2 : i >> 1) * 16 * row_bytes);
  }
};

// A descriptor of `bytes` from p on; everything in it is uniform, which the
// compiler has to be told of what was divided.
__device__ __forceinline__ int64_t uniform(int64_t v) {
  return (int64_t)(((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32) |
                   (uint32_t)__builtin_amdgcn_readfirstlane((int)v));
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t mm_rsrc(const char* p, int64_t bytes) {
  const int64_t cap = 0x7FFFFFFF;
  const int size = (int)(bytes < 0 ? 0 : bytes < cap ? bytes : cap);
  return __builtin_amdgcn_make_buffer_rsrc(
      reinterpret_cast<char*>(uniform(reinterpret_cast<int64_t>(p))), 0,
      __builtin_amdgcn_readfirstlane(size), 0x00020000);
}

// The transposing read behind a pointer of its own: without that scope the
// compiler takes the read for one of what the loads to LDS still bring, and waits
// for all of them (8192^3, both operands k-major: 1070 TFLOP/s without the wait).
// The kernel waits for them itself.
__device__ __forceinline__ u32x2_t mm_read_tr16(const char* __restrict__ p) {
  return lds_read_tr16(p);
}

// Tile `at` of job ji: its slabs and its epilogue.  AKM, BKM: the operand is
// k-major.  PAIR: A's rows alternate in groups of 16 between a and a2 (a tile has
// TM / 2 features of each).
template <bool AKM, bool BKM, bool PAIR, class Sh, class Epi>
__device__ __forceinline__ void mm_tile(const MmArgs& args, const typename Epi::Args& ea,
                                        char* smem, int ji, int at) {
  constexpr int TM = Sh::TM, TN = Sh::TN, TI = Sh::TI, TJ = Sh::TJ;
  constexpr int QA = Sh::A_BYTES / 1024 / Sh::WAVES, QB = Sh::B_BYTES / 1024 / Sh::WAVES;
  static_assert(!PAIR || (!AKM && QA % 4 == 0), "paired rows");
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / Sh::WN, wn = wave % Sh::WN;

  constexpr int STAGE_A = Sh::A_BYTES, STAGE_B = Sh::B_BYTES;
  char* const lds_a = smem + wave * QA * 1024;
  char* const lds_b = smem + 2 * STAGE_A + wave * QB * 1024;
  // (what follows is uniform; the compiler has to be told of what was loaded or
  // divided)
  const MmJob& job = args.job[ji];
  const int n_all = __builtin_amdgcn_readfirstlane(job.n_rows ? *job.n_rows : job.n);
  const int k_all = __builtin_amdgcn_readfirstlane(job.k_rows ? *job.k_rows : job.k);
  const int m_all = job.m, m_tiles = job.m_tiles;
  const int n_tiles = job.n_rows ? (n_all + TN - 1) / TN : job.n_tiles;
  // Blocks go round the 8 XCDs: each gets a run of neighbouring tiles, in
  // groups of 4 tiles along n, so that its L2 holds what they share.
  const int total = m_tiles * n_tiles * job.splits;
  at -= job.block0;
  if (at >= total) return;
  {
    const int x = at & 7, q = total >> 3, r = total & 7;
    at = x * q + (x < r ? x : r) + (at >> 3);
  }
  const int split = __builtin_amdgcn_readfirstlane(at / (m_tiles * n_tiles));
  at -= split * m_tiles * n_tiles;
  const int g0 = __builtin_amdgcn_readfirstlane(at / (4 * m_tiles)) * 4;
  const int gn = n_tiles - g0 < 4 ? n_tiles - g0 : 4;
  at -= g0 * m_tiles;
  const int mt = __builtin_amdgcn_readfirstlane(at / gn);
  constexpr int A_TILE = PAIR ? TM / 2 : TM;
  const int m0 = mt * A_TILE, n0 = (g0 + at - mt * gn) * TN;
  const int64_t lda = job.lda * 2, ldb = job.ldb * 2;
  const int a_rows = m_all - m0 < A_TILE ? m_all - m0 : A_TILE;
  const int b_rows = n_all - n0 < TN ? n_all - n0 : TN;
  const int m_end = (m_all - m0 + 7) & ~7, n_end = (n_all - n0 + 7) & ~7;
  const int64_t a0 = AKM ? (int64_t)m0 * 2 : m0 * lda, b0 = BKM ? (int64_t)n0 * 2 : n0 * ldb;
  const char *pa = job.a + a0, *pa2 = job.a2 + a0, *pb = job.b + b0;
  const int64_t a_plane = job.a_plane, b_plane = job.b_plane;
  const int64_t a_part = job.a_part, b_part = job.b_part;
  MmSource<AKM, PAIR> sa;
  MmSource<BKM, false> sb;
  sa.place(lane, job.lda);
  sb.place(lane, job.ldb);
  const int pairs = job.pairs, code = job.code, per_seg = (k_all + kSlab - 1) / kSlab;
  const int all = per_seg * pairs * job.parts;
  const int per = __builtin_amdgcn_readfirstlane((all + job.splits - 1) / job.splits);
  const int s0 = split * per;
  const int slabs = __builtin_amdgcn_readfirstlane((s0 + per < all ? s0 + per : all) - s0);
  // the next slab to load: its segment and first k
  int to_load = slabs, seg = __builtin_amdgcn_readfirstlane(slabs > 0 ? s0 / per_seg : 0);
  int k0 = (s0 - seg * per_seg) * kSlab;

  __amdgpu_buffer_rsrc_t ra, ra2, rb;
  uint32_t oa[2], ob[2];
  // What the next slab's loads need, and the loads.  Past the last slab the
  // descriptors are empty, and zeros come.
  auto aim = [&]() SM_INLINE {
    const int left = k_all - k0, rows = left < kSlab ? left : kSlab;
    const int part = seg >= pairs ? 1 : 0, pair = seg - part * pairs;
    const int pl = code >> (4 * pair);
    const int64_t a_at = (pl & 3) * a_plane + part * a_part + (AKM ? k0 * lda : (int64_t)k0 * 2);
    const int64_t b_at =
        (pl >> 2 & 3) * b_plane + part * b_part + (BKM ? k0 * ldb : (int64_t)k0 * 2);
    // bytes from the slab's base to the end of what may be read
    const int64_t a_end = AKM ? (rows - 1) * lda + m_end * 2
                              : (a_rows - 1) * lda + ((left + 7) & ~7) * 2;
    const int64_t b_end = BKM ? (rows - 1) * ldb + n_end * 2
                              : (b_rows - 1) * ldb + ((left + 7) & ~7) * 2;
    ra = mm_rsrc(pa + a_at, to_load > 0 ? a_end : 0);
    if constexpr (PAIR) ra2 = mm_rsrc(pa2 + a_at, to_load > 0 ? a_end : 0);
    rb = mm_rsrc(pb + b_at, to_load > 0 ? b_end : 0);
    sa.slab(left, oa);
    sb.slab(left, ob);
    --to_load;
    k0 += kSlab;
    if (k0 >= k_all) k0 = 0, ++seg;
  };
  auto fire = [&](int stage) SM_INLINE {
#pragma unroll
    for (int q = 0; q < QA; ++q)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(PAIR && (q >> 1 & 1) ? ra2 : ra,
                                               (lds_void*)(lds_a + stage * STAGE_A + q * 1024), 16,
                                               sa.at(oa, wave * QA + q), 0, 0, 0);
#pragma unroll
    for (int q = 0; q < QB; ++q)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb,
                                               (lds_void*)(lds_b + stage * STAGE_B + q * 1024), 16,
                                               sb.at(ob, wave * QB + q), 0, 0, 0);
  };

  // A fragment of MFMA tile t (16 rows from the wave's first) and k-step kk.
  // k along rows: one 16-byte read.  k-major: two transposing reads, 4 rows
  // apart, as in the layout's comment; the wave's columns begin at c0.
  constexpr int RA = TM / Sh::WM, RB = TN / Sh::WN;
  const int fa = AKM ? (wm * RA >> 7) * 16384 +
                           km_off<bf16_t>(8 * (lane >> 4) + ((lane & 15) >> 2),
                                          2 * (wm * RA & 127) + 8 * (lane & 3))
                     : lds_off<128>(wm * RA + (lane & 15), lane >> 4);
  const int fb = 2 * STAGE_A +
                 (BKM ? (wn * RB >> 7) * 16384 +
                            km_off<bf16_t>(8 * (lane >> 4) + ((lane & 15) >> 2),
                                           2 * (wn * RB & 127) + 8 * (lane & 3))
                      : lds_off<128>(wn * RB + (lane & 15), lane >> 4));
  auto frag = [&](auto km, int base, int stage_at, int t, int kk) SM_INLINE -> bf16x8_t {
    if constexpr (decltype(km)::value) {
      const char* p = smem + (base ^ (t << 5)) + stage_at + kk * 8192;
      const u32x2_t lo = mm_read_tr16(p), hi = mm_read_tr16(p + 1024);
      return __builtin_bit_cast(bf16x8_t, u32x4_t{lo[0], lo[1], hi[0], hi[1]});
    } else {
      return *reinterpret_cast<const bf16x8_t*>(smem + (base ^ (kk << 6)) + stage_at + t * 2048);
    }
  };

  f32x4_t acc[TI][TJ];
  // A slab goes in steps: its two k-steps of 32, by parts of A's rows.  While one
  // is multiplied the fragments of the next are read.  The next slab is waited for
  // before the last step: past that barrier every wave has read all of this slab,
  // whose place the loads of the slab after next then take.  (Quarters of a
  // k-major A of 128 rows: its addresses take the registers that halves would
  // need, and a register spilled to memory waits for all loads to LDS.)
  constexpr int NQ = AKM && TI == 8 ? 4 : 2, HI = TI / NQ;
  bf16x8_t a[2][HI], b[2][TJ];
  auto read_a = [&](int stage, auto kk, auto part) SM_INLINE {
    constexpr int K = decltype(kk)::value, H = decltype(part)::value;
#pragma unroll
    for (int i = 0; i < HI; ++i)
      a[H & 1][i] = frag(std::bool_constant<AKM>{}, fa, stage * STAGE_A, H * HI + i, K);
  };
  auto read_b = [&](int stage, auto kk) SM_INLINE {
    constexpr int K = decltype(kk)::value;
#pragma unroll
    for (int j = 0; j < TJ; ++j)
      b[K][j] = frag(std::bool_constant<BKM>{}, fb, stage * STAGE_B, j, K);
  };
  constexpr std::integral_constant<int, 0> c0{};
  constexpr std::integral_constant<int, 1> c1{};
  constexpr int RDA = HI * (AKM ? 2 : 1), RDB = TJ * (BKM ? 2 : 1);
  // the products of a step, in this order: `reads` reads first, `loads` loads among
  // the products
  auto multiply = [&](auto kk, auto part, auto reads, auto loads) SM_INLINE {
    constexpr int K = decltype(kk)::value, H = decltype(part)::value;
    constexpr int R = decltype(reads)::value, L = decltype(loads)::value;
#pragma unroll
    for (int i = 0; i < HI; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j)
        acc[H * HI + i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            a[H & 1][i], b[K][j], acc[H * HI + i][j], 0, 0, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, R, 0);
    if constexpr (L == 0) {
      __builtin_amdgcn_sched_group_barrier(0x008, HI * TJ, 0);
    } else {
#pragma unroll
      for (int l = 0; l < L; ++l) {
        __builtin_amdgcn_sched_group_barrier(0x008, HI * TJ / L, 0);
        __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto parts_of = [&](int stage, auto kk, auto self, auto part) SM_INLINE {
    constexpr int H = decltype(part)::value;
    if constexpr (H + 1 < NQ) {
      constexpr std::integral_constant<int, H + 1> next{};
      read_a(stage, kk, next);
      multiply(kk, part, std::integral_constant<int, RDA>{}, c0);
      self(stage, kk, self, next);
    }
  };
  auto slab = [&](int stage) SM_INLINE {
    constexpr std::integral_constant<int, NQ - 1> end{};
    parts_of(stage, c0, parts_of, c0);
    read_b(stage, c1);
    read_a(stage, c1, c0);
    aim();
    multiply(c0, end, std::integral_constant<int, RDA + RDB>{}, c0);
    parts_of(stage, c1, parts_of, c0);
    wait_vmcnt<0>();
    wait_lgkmcnt0();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read_b(stage ^ 1, c0);
    read_a(stage ^ 1, c0, c0);
    fire(stage);
    multiply(c1, end, std::integral_constant<int, RDA + RDB>{},
             std::integral_constant<int, QA + QB>{});
  };
  aim();
  fire(0);
  aim();
  fire(1);
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  wait_vmcnt<QA + QB>();
  __builtin_amdgcn_s_barrier();
  read_b(0, c0);
  read_a(0, c0, c0);
  // (an odd slab too many is zeros)
  for (int s = 0; s < slabs; s += 2) {
    slab(0);
    slab(1);
  }
  // the last, empty loads: the epilogue's LDS, and the block's end, wait for them
  wait_vmcnt<0>();
  __builtin_amdgcn_s_barrier();
  // (opaque, so that the epilogue's addresses are not held through the loop)
  int lane_after = lane;
  asm volatile("" : "+v"(lane_after));
  Epi::template run<TI, TJ>(ea,
                            MmPlace{ji, split, m0 + wm * (PAIR ? RA / 2 : RA), n0 + wn * RB, m_all,
                                    n_all, lane_after, smem + wave * (Sh::LDS / Sh::WAVES)},
                            acc);
}

__device__ __forceinline__ int mm_job(const MmArgs& args, int at) {
  int ji = 0;
#pragma unroll
  for (int i = 1; i < kMaxJobs; ++i)
    if (i < args.jobs && at >= args.job[i].block0) ji = i;
  return ji;
}

// (The kernels' buffer instructions are unknown to the host's pass.)
template <bool AKM, bool BKM, bool PAIR, class Sh, class Epi>
__global__ __launch_bounds__(64 * Sh::WAVES, Sh::WPE) void k_mm(MmArgs args,
                                                                typename Epi::Args ea) {
#ifdef __HIP_DEVICE_COMPILE__
  __shared__ __align__(1024) char smem[Sh::LDS];
  mm_tile<AKM, BKM, PAIR, Sh, Epi>(args, ea, smem, mm_job(args, blockIdx.x), blockIdx.x);
#endif
}
// A k-major, B of either kind: products whose tiles share the chip.
template <class Sh, class Epi>
__global__ __launch_bounds__(64 * Sh::WAVES, Sh::WPE) void k_mm_both(MmArgs args,
                                                                     typename Epi::Args ea) {
#ifdef __HIP_DEVICE_COMPILE__
  __shared__ __align__(1024) char smem[Sh::LDS];
  const int ji = __builtin_amdgcn_readfirstlane(mm_job(args, blockIdx.x));
  if (args.job[ji].b_km) mm_tile<true, true, false, Sh, Epi>(args, ea, smem, ji, blockIdx.x);
  else mm_tile<true, false, false, Sh, Epi>(args, ea, smem, ji, blockIdx.x);
#endif
}

}  // namespace sm
