// Operand copies of the matrix products and the join of split sums.
#include "sm_mm_ops.h"

namespace sm {

// The job of a block, and the block's place in it.
template <int MAX>
__device__ __forceinline__ int job_of(const int32_t (&block0)[MAX], int jobs, int& block) {
  int ji = 0;
#pragma unroll
  for (int i = 1; i < MAX; ++i)
    if (i < jobs && (int)blockIdx.x >= block0[i]) ji = i;
  block = blockIdx.x - block0[ji];
  return ji;
}
// Blocks of 256 threads for `work` pieces, about 8 pieces a thread where there are
// many.
int64_t copy_blocks(int64_t work) {
  const int64_t b = (work + 255) / 256;
  return b <= 2048 ? b : std::max<int64_t>(2048, b / 8);
}

// A thread copies 8 entries of a row.  Bound by HBM.
template <typename T, int P>
__global__ __launch_bounds__(256) void k_planes(PlanesJobs all) {
  int block;
  const int ji = job_of(all.block0, all.jobs, block);
  const PlanesArgs& a = all.job[ji];
  const int blocks = (ji + 1 < all.jobs ? all.block0[ji + 1] : (int)gridDim.x) - all.block0[ji];
  const T* src = static_cast<const T*>(a.src);
  const int64_t live = a.count ? *a.count : a.rows, plane = a.rows * a.ld;
  const int per = a.ld / 8, cols = a.cols;
  for (int64_t i = (int64_t)block * 256 + threadIdx.x; i < live * per; i += (int64_t)blocks * 256) {
    const int64_t r = i / per;
    const int c = (int)(i - r * per) * 8;
    const T* p = src + (a.list ? (int64_t)a.list[r] : r) * a.stride + c;
    float v[8];
    if (c + 8 <= cols) {
      Piece<T, 8> in;
      in.load(p);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = in[k];
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = c + k < cols ? to_f32(p[k]) : 0.f;
    }
    store_mid<P>(a.dst + r * a.ld + c, plane, f32x4_t{v[0], v[1], v[2], v[3]});
    store_mid<P>(a.dst + r * a.ld + c + 4, plane, f32x4_t{v[4], v[5], v[6], v[7]});
  }
}

hipError_t launch_planes(PlanesJobs& a, int32_t dtype, hipStream_t s) {
  int64_t blocks = 0;
  for (int i = 0; i < a.jobs; ++i) {
    a.block0[i] = (int)blocks;
    blocks += copy_blocks(a.job[i].rows * (a.job[i].ld / 8));
    if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  }
  if (blocks == 0) return hipSuccess;
  if (dtype == SM_BF16)
    hipLaunchKernelGGL((k_planes<bf16_t, 1>), dim3((unsigned)blocks), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((k_planes<float, 3>), dim3((unsigned)blocks), dim3(256), 0, s, a);
  return hipGetLastError();
}

// A thread joins 4 entries of a row, in the order of the splits.
template <typename T>
__device__ __forceinline__ void join_rows(const JoinArgs& a, int block, int blocks) {
  const int per = (a.cols + 3) / 4;
  for (int64_t i = (int64_t)block * 256 + threadIdx.x; i < a.rows * per;
       i += (int64_t)blocks * 256) {
    const int64_t r = i / per;
    const int c = (int)(i - r * per) * 4, here = a.cols - c;
    const int64_t at = a.pos ? a.pos[r] : r;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (at >= 0) {
      const float* p = a.part + at * a.part_ld + c;
      for (int k = 0; k < a.splits; ++k, p += a.split_step) {
        const f32x4_t t = *reinterpret_cast<const f32x4_t*>(p);
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] += t[q];
      }
    }
    if (a.by && at >= 0) {       // (a factor that is not finite leaves zeros alone)
      const float by = *a.by;
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] *= by;
    }
    T* o = static_cast<T*>(a.out) + r * a.ld + c;
    if (a.add) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (q < here) v[q] += to_f32(o[q]);
    }
    if (here >= 4) {
      store_vec<4>(o, v);
    } else {
      for (int q = 0; q < here; ++q) put(o + q, v[q]);
    }
  }
}
__global__ __launch_bounds__(256) void k_join(JoinJobs all) {
  int block;
  const int ji = job_of(all.block0, all.jobs, block);
  const JoinArgs& a = all.job[ji];
  const int blocks = (ji + 1 < all.jobs ? all.block0[ji + 1] : (int)gridDim.x) - all.block0[ji];
  if (a.dtype == SM_BF16) join_rows<bf16_t>(a, block, blocks);
  else join_rows<float>(a, block, blocks);
}

namespace {

// When the blocks of the jobs are done, in microseconds: `len` a block of each job,
// dealt out in order to `slots` places as they fall free.  Places are kept as
// levels, equal ones together.
double makespan(const int64_t* blocks, const double* len, int jobs, int slots) {
  struct Level {
    double t;
    int64_t c;
  } lv[64];
  int n = 1;
  lv[0] = {0.0, slots};
  double last = 0.0;
  for (int j = 0; j < jobs; ++j) {
    int64_t left = blocks[j];
    // whole rounds over all places change nothing but the time
    if (left > 8 * slots) {
      const int64_t rounds = left / slots - 7;
      for (int i = 0; i < n; ++i) lv[i].t += rounds * len[j];
      left -= rounds * slots;
    }
    while (left > 0) {
      int lo = 0;
      for (int i = 1; i < n; ++i)
        if (lv[i].t < lv[lo].t) lo = i;
      const int64_t k = std::min(left, lv[lo].c);
      const double t = lv[lo].t + len[j];
      left -= k;
      lv[lo].c -= k;
      if (lv[lo].c == 0) lv[lo] = lv[--n];
      int at = 0;
      while (at < n && lv[at].t != t) ++at;
      if (at < n) lv[at].c += k;
      else if (n < 64) lv[n++] = {t, k};
      else lv[0].c += k;      // (no more than an estimate)
    }
  }
  for (int i = 0; i < n; ++i) last = std::max(last, lv[i].t);
  return last;
}

}  // namespace

MmPlan plan_products(const MmSize* sizes, int jobs) {
  MmPlan best{};
  double least = 1e30;
  for (const bool wide : {true, false}) {
    const int t = wide ? 256 : 128, slots = wide ? kCus : 2 * kCus;
    const double slab = wide ? 1.65 : 1.0;
    int64_t longest = 1;
    for (int j = 0; j < jobs; ++j) longest = std::max(longest, sizes[j].slabs);
    for (int part = 1; part <= 16; ++part) {
      const double target = (double)longest / part;
      if (part > 1 && target < 4) break;
      MmPlan p{};
      p.wide = wide;
      int64_t blocks[kMaxJobs];
      double len[kMaxJobs], cost = 0;
      bool split = false;
      for (int j = 0; j < jobs; ++j) {
        const MmSize& z = sizes[j];
        const int64_t tiles = ((z.m + t - 1) / t) * ((z.n + t - 1) / t);
        const int64_t most = z.may_split ? std::min<int64_t>(16, std::max<int64_t>(1, z.slabs / 4))
                                         : 1;
        p.splits[j] =
            (int)std::max<int64_t>(1, std::min<int64_t>(most, (int64_t)(z.slabs / target + 0.5)));
        split = split || p.splits[j] > 1;
        blocks[j] = tiles * p.splits[j];
        len[j] = slab * ((z.slabs + p.splits[j] - 1) / p.splits[j]) + 5.0;
        // the sums are written and read (4 bytes, at about 5 MB a microsecond), by a
        // launch of their own
        if (p.splits[j] > 1) cost += p.splits[j] * z.m * z.n * 8 / 5e6;
      }
      if (part > 1 && !split) continue;
      // longest first, as they are launched
      for (int i = 0; i < jobs; ++i)
        for (int j = i + 1; j < jobs; ++j)
          if (len[j] > len[i]) std::swap(len[i], len[j]), std::swap(blocks[i], blocks[j]);
      cost += makespan(blocks, len, jobs, slots) + (split ? 5.0 : 0.0);
      if (cost < least) least = cost, best = p;
    }
  }
  return best;
}

void MmStores::add(const MmJob& j, bool b_km, void* dst, int32_t dtype, int32_t accumulate,
                   float* sums, int splits, const float* by) {
  const int i = a.jobs++;
  a.job[i] = j;
  a.job[i].b_km = b_km;
  a.job[i].splits = splits;
  const int64_t ld = round_up(j.m, 4);
  join.job[i] = JoinArgs{};
  if (splits > 1) {
    e.out[i] = sums_out(sums, j.m, j.n);
    join.job[i] = {sums, j.n * ld, ld, splits, nullptr, j.n, j.m, dtype, accumulate, dst, j.m, by};
  } else {
    e.out[i] = {dst, j.m, 0, dtype, accumulate, by};
  }
}

hipError_t MmStores::run(bool wide, hipStream_t s) {
  if (a.jobs == 0) return hipSuccess;
  // the longest blocks first
  const auto length = [&](const MmJob& j) {
    return (int64_t)j.k * j.pairs * j.parts / j.splits;
  };
  bool km = false, rows = false;
  for (int i = 0; i < a.jobs; ++i) {
    for (int k = i + 1; k < a.jobs; ++k)
      if (length(a.job[k]) > length(a.job[i])) {
        std::swap(a.job[i], a.job[k]);
        std::swap(e.out[i], e.out[k]);
        std::swap(join.job[i], join.job[k]);
      }
    (a.job[i].b_km ? km : rows) = true;
  }
  const auto go = [&](auto shape) {
    typedef decltype(shape) Sh;
    return km ? run_mm_as<true, true, false, Sh, EpiStore>(a, e, rows, s)
              : run_mm_as<true, false, false, Sh, EpiStore>(a, e, false, s);
  };
  SM_TRY(wide ? go(MmShape<256, 256, 2, 4>{}) : go(MmShape<128, 128, 2, 2>{}));
  return joins(s);
}

hipError_t MmStores::joins(hipStream_t s) {
  JoinJobs j{};
  for (int i = 0; i < a.jobs; ++i)
    if (join.job[i].splits > 0) j.job[j.jobs++] = join.job[i];
  return launch_join(j, s);
}

hipError_t launch_join(JoinJobs& a, hipStream_t s) {
  int64_t blocks = 0;
  for (int i = 0; i < a.jobs; ++i) {
    a.block0[i] = (int)blocks;
    blocks += copy_blocks(a.job[i].rows * ((a.job[i].cols + 3) / 4));
    if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  }
  if (blocks == 0) return hipSuccess;
  hipLaunchKernelGGL(k_join, dim3((unsigned)blocks), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <typename T>
__global__ __launch_bounds__(256) void k_zero(T* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    p[i] = 0;
}

hipError_t launch_zero(void* p, int32_t dtype, int64_t n, hipStream_t s) {
  if (n == 0) return hipSuccess;
  const dim3 grid((unsigned)std::min<int64_t>((n + 255) / 256, 4096));
  if (dtype == SM_BF16) hipLaunchKernelGGL(k_zero<bf16_t>, grid, dim3(256), 0, s, (bf16_t*)p, n);
  else hipLaunchKernelGGL(k_zero<uint32_t>, grid, dim3(256), 0, s, (uint32_t*)p, n);
  return hipGetLastError();
}

}  // namespace sm
