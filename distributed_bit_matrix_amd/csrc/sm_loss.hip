// Softmax cross entropy of a linear output layer (signmuon_layers.h), forward
// and backward, without the logits in memory.
//
// Rows to be ignored leave first: their targets and activations are gathered
// out, so they cost no product, and whatever they hold reaches no gradient.
// The number of rows left stays on the device; the products' tiles past it end
// at once.
//
// Forward: the product's epilogue keeps of a tile of logits each row's maximum
// and sum of exponentials over the wave's 128 features, and the target's logit;
// one launch joins them.  Backward, in pieces of the vocabulary: the logits of a
// piece again, with G = (softmax - onehot) * upstream written by the epilogue
// (the softmax's statistics are known), then dX += G W and dW = G^T X of it.
// Where the logits make few tiles (a small vocabulary), their product's k is
// split, and a launch of its own does what the epilogues do.
//
// G is rounded to the operands' precision: for bfloat16 half a step of 2^-8 an
// entry, as much as the rounding of the gradients themselves, where errors
// average.  A row's gradient is mostly its target's entry, so over few rows, or
// few results, they do not: there G has two bfloat16 planes.  An upstream factor
// that all rows share would be rounded alike in all of them: it is left out of G
// and multiplies the results.
//
// 11059 of 12288 rows against 50257 x 768 bfloat16: the logits' launch 912 us (940
// TFLOP/s; a tile has 12 slabs, and its first loads and epilogue, with nothing
// beside them in a CU that holds one block, are a third of it); backward 2 pieces,
// 502 and 475 us for the logits and G, 806 and 827 for the two products (1060
// TFLOP/s).
#include <cmath>

#include "sm_few.h"
#include "sm_layers.h"
#include "sm_mm_ops.h"
#include "sm_thin.h"

namespace sm {

constexpr float kLog2e = 1.44269504088896341f;

// ---------------------------------------------------------------------------
// The list of rows that count, in order: list[i] the row, target[i] its target,
// pos[r] its place or -1.  One block, 1024 rows a step: 12288 rows take 12
// steps of a ballot and a sum over waves.
// ---------------------------------------------------------------------------
template <typename I>
__global__ __launch_bounds__(1024) void k_loss_list(const I* targets, int rows, int64_t ignore,
                                                    int32_t* list, int32_t* target, int32_t* pos,
                                                    int32_t* count, int vocab) {
  __shared__ int sums[2][16];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int base = 0, turn = 0;
  for (int r0 = 0; r0 < rows; r0 += 1024, turn ^= 1) {
    const int r = r0 + threadIdx.x;
    const int64_t t = r < rows ? (int64_t)targets[r] : ignore;
    const bool keep = r < rows && t != ignore;
    const uint64_t b = __ballot(keep);
    if (lane == 0) sums[turn][w] = __popcll(b);
    __syncthreads();
    int before = base, all = base;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      if (k < w) before += sums[turn][k];
      all += sums[turn][k];
    }
    const int at = before + __popcll(b & (((uint64_t)1 << lane) - 1));
    if (keep) {
      list[at] = r;
      target[at] = t >= 0 && t < vocab ? (int)t : -1;    // -1: no such entry
    }
    if (r < rows) pos[r] = keep ? at : -1;
    base = all;
  }
  if (threadIdx.x == 0) *count = base;
}

// ---------------------------------------------------------------------------
// Epilogues
// ---------------------------------------------------------------------------
// Per row and 128 (or 64) features: maximum and sum of exp(z - maximum); the
// target's logit.  part: [strip][cap], strips of TI * 16 features.
struct EpiLse {
  struct Args {
    float2* part;
    int64_t cap;
    const int32_t* target;
    float* picked;
  };
  template <bool WHOLE, int TI, int TJ>
  static __device__ __forceinline__ void rows(const Args& e, const MmPlace& at,
                                              const f32x4_t (&acc)[TI][TJ]) {
    const int mc = at.m0 + 4 * (at.lane >> 4), nc = at.n0 + (at.lane & 15);
    const int64_t strip = at.m0 / (TI * 16);
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const int n = nc + 16 * j;
      float mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (WHOLE || mc + 16 * i + k < at.m) mx = fmaxf(mx, acc[i][j][k]);
      mx = fmaxf(mx, __shfl_xor(mx, 16));
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      // The largest logit's own term is 1 to the last bit: where the target has it the
      // loss is the logarithm of the sum alone, and a rounding of mx log2(e) (one
      // multiply-add a logit, 821 us a call of the size above instead of 832) would be
      // all of it, of either sign.
      const float ref = mx == -INFINITY ? 0.f : mx;
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float p = __builtin_amdgcn_exp2f((acc[i][j][k] - ref) * kLog2e);
          s += WHOLE || mc + 16 * i + k < at.m ? p : 0.f;
        }
      s += __shfl_xor(s, 16);
      s += __shfl_xor(s, 32);
      const int t = n < at.n ? e.target[n] : -1;
      const bool mine = t >= at.m0 && t < at.m0 + TI * 16 && ((t >> 2) & 3) == at.lane >> 4;
      if (__any(mine)) {       // of a vocabulary's strips few have the target
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) z = mc + 16 * i + k == t ? acc[i][j][k] : z;
        if (mine) e.picked[n] = z;
      }
      if (n < at.n && at.lane < 16) e.part[strip * e.cap + n] = make_float2(mx, s);
    }
  }
  template <int TI, int TJ>
  static __device__ __forceinline__ void run(const Args& e, const MmPlace& at,
                                             const f32x4_t (&acc)[TI][TJ]) {
    if (at.m0 + TI * 16 <= at.m) rows<true>(e, at, acc);
    else if (at.m0 < at.m) rows<false>(e, at, acc);
  }
};

// The same for few rows, which are all there (an ignored one is left out by the
// join): a wave's strip is all groups of 16 features that it had.  part:
// [row][strips].
template <typename T>
struct FewLse {
  struct Args {
    float2* part;
    int32_t strips;
    const void* targets;
    int32_t target_bits;
    float* picked;
  };
  Args e;
  int lane, n;
  int64_t t;
  float m = -INFINITY, s = 0.f;
  __device__ __forceinline__ FewLse(const Args& a, int l, int rows) : e(a), lane(l), n(rows) {
    const int r = (l & 15) < rows ? l & 15 : rows - 1;
    t = a.target_bits == 64 ? static_cast<const int64_t*>(a.targets)[r]
                            : static_cast<const int32_t*>(a.targets)[r];
  }
  __device__ __forceinline__ void group(int m0, int all, const f32x4_t (&acc)[1]) {
    const int f = m0 + 4 * (lane >> 4);
    float top = m;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (f + k < all) top = fmaxf(top, acc[0][k]);
      if (f + k == t && (lane & 15) < n) e.picked[lane & 15] = acc[0][k];
    }
    const float ref = top == -INFINITY ? 0.f : top;
    s *= __builtin_amdgcn_exp2f((m - ref) * kLog2e);      // (0 where m is -inf)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (f + k < all) s += __builtin_amdgcn_exp2f((acc[0][k] - ref) * kLog2e);
    m = top;
  }
  __device__ __forceinline__ void finish(int wave) {
#pragma unroll
    for (int o = 16; o < 64; o *= 2) {
      const float mo = __shfl_xor(m, o), so = __shfl_xor(s, o), top = fmaxf(m, mo);
      const float ref = top == -INFINITY ? 0.f : top;
      s = s * __builtin_amdgcn_exp2f((m - ref) * kLog2e) +
          so * __builtin_amdgcn_exp2f((mo - ref) * kLog2e);
      m = top;
    }
    if (lane < n) e.part[lane * e.strips + wave] = make_float2(m, s);
  }
};

// G = (exp(z - lse) - onehot) * scale of a piece of the vocabulary that begins
// at v0: to planes of [rows][ld].
template <int P>
struct EpiGrad {
  struct Args {
    bf16_t* g;
    int64_t ld, plane;
    int32_t v0;
    const int32_t* target;
    const float *lse, *scale;
  };
  template <bool WHOLE, int TI, int TJ>
  static __device__ __forceinline__ void rows(const Args& e, const MmPlace& at,
                                              const f32x4_t (&acc)[TI][TJ]) {
    const int mc = at.m0 + 4 * (at.lane >> 4), nc = at.n0 + (at.lane & 15);
    const int cols = ((at.m + 7) & ~7) - at.m0;      // zeros up to a whole piece of 16 bytes
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const int n = nc + 16 * j, r = n < at.n ? n : at.n - 1;
      const int t = e.target[r] - e.v0;
      const float scale = e.scale[r];
      // (the difference first: lse log2(e) may be past float32's range)
      const float lse = e.lse[r];
      f32x4_t v[TI];
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float p = __builtin_amdgcn_exp2f((acc[i][j][k] - lse) * kLog2e) * scale;
          v[i][k] = WHOLE || mc + 16 * i + k < at.m ? p : 0.f;
        }
      if (__any(t >= at.m0 && t < at.m0 + TI * 16)) {
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (mc + 16 * i + k == t) {
              const float p = __builtin_amdgcn_exp2f((acc[i][j][k] - lse) * kLog2e);
              v[i][k] = (p - 1.f) * scale;
            }
      }
      const int n0 = at.n0 + 16 * j;
      put_planes<P, 16 * TI>(at, v, e.g + (int64_t)n0 * e.ld + at.m0, e.plane, e.ld, at.n - n0,
                             cols);
    }
  }
  template <int TI, int TJ>
  static __device__ __forceinline__ void run(const Args& e, const MmPlace& at,
                                             const f32x4_t (&acc)[TI][TJ]) {
    if (at.m0 + TI * 16 <= at.m) rows<true>(e, at, acc);
    else rows<false>(e, at, acc);
  }
};

// What EpiLse does, where the logits are sums of splits: [split][rows][vocab rounded
// up to 4].  A wave has a row's strip of kMidStrip logits.
constexpr int kMidStrip = 1024;
__global__ __launch_bounds__(256) void k_loss_mid(const float* sums, int splits,
                                                  const int32_t* count, int rows, int vocab,
                                                  int strips, EpiLse::Args e) {
  constexpr int V = kMidStrip / 256;
  const int lane = threadIdx.x & 63;
  const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int n = (int)(i / strips), strip = (int)(i - (int64_t)n * strips);
  if (n >= *count) return;
  const int64_t ld = (vocab + 3) & ~3;
  const float* p = sums + n * ld;
  f32x4_t z[V];
#pragma unroll
  for (int v = 0; v < V; ++v) z[v] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int k = 0; k < splits; ++k, p += rows * ld) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = strip * kMidStrip + 256 * v + 4 * lane;
      if (c < vocab) z[v] += *reinterpret_cast<const f32x4_t*>(p + c);
    }
  }
  const int t = e.target[n];
  float m = -INFINITY;
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = strip * kMidStrip + 256 * v + 4 * lane + k;
      if (c < vocab) m = fmaxf(m, z[v][k]);
      if (c == t) e.picked[n] = z[v][k];
    }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
  const float ref = m == -INFINITY ? 0.f : m;
  float s = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (strip * kMidStrip + 256 * v + 4 * lane + k < vocab)
        s += __builtin_amdgcn_exp2f((z[v][k] - ref) * kLog2e);
  s = lanes_sum<64>(s);
  if (lane == 0) e.part[strip * e.cap + n] = make_float2(m, s);
}

// ---------------------------------------------------------------------------
// Forward: the strips' sums joined, 16 rows by 64 lanes over the strips.
// loss[r], lse[r] of the caller's rows; a row whose target does not exist has
// a NaN for its loss.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(1024) void k_loss_join(const float2* part, int64_t cap, int strips,
                                                    const int32_t* count, const int32_t* list,
                                                    const int32_t* target, const float* picked,
                                                    float* loss, float* lse) {
  __shared__ float2 sh[64][17];
  const int x = threadIdx.x & 15, y = threadIdx.x >> 4;
  const int n = blockIdx.x * 16 + x, live = *count;
  if (blockIdx.x * 16 >= live) return;
  float m = -INFINITY, s = 0.f;
  if (n < live) {
#pragma unroll 4
    for (int k = y; k < strips; k += 64) {
      const float2 v = part[k * cap + n];
      const float top = fmaxf(m, v.x);
      if (top == -INFINITY) {
        s += v.y;
      } else {
        s = s * __builtin_amdgcn_exp2f((m - top) * kLog2e) +
            v.y * __builtin_amdgcn_exp2f((v.x - top) * kLog2e);
        m = top;
      }
    }
  }
  sh[y][x] = make_float2(m, s);
  __syncthreads();
  // a wave joins one row
  const int row = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const float2 v = sh[lane][row];
  float top = v.x;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
  float t = v.y;
  if (v.x != -INFINITY) t *= __builtin_amdgcn_exp2f((v.x - top) * kLog2e);
  t = lanes_sum<64>(t);
  const int at = blockIdx.x * 16 + row;
  if (lane == 0 && at < live) {
    const float ln = logf(t);
    const int r = list[at];
    lse[r] = top + ln;
    loss[r] = target[at] < 0 ? NAN : top - picked[at] + ln;
  }
}

// G from such sums; a thread has 4 entries of a row, the last of a row's 8 zero.
template <int P>
__global__ __launch_bounds__(256) void k_loss_mid_grad(const float* sums, int splits,
                                                       const int32_t* count, int rows, int cols,
                                                       const int32_t* target, int v0,
                                                       const float* lse, const float* scale,
                                                       bf16_t* g, int64_t g_ld, int64_t plane) {
  const int per = ((cols + 7) & ~7) / 4;
  const int64_t ld = (cols + 3) & ~3, all = (int64_t)*count * per;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all;
       i += (int64_t)gridDim.x * 256) {
    const int r = (int)(i / per), c = (int)(i - (int64_t)r * per) * 4;
    f32x4_t z = {0.f, 0.f, 0.f, 0.f};
    if (c < cols) {
      const float* p = sums + r * ld + c;
#pragma unroll 4
      for (int k = 0; k < splits; ++k, p += rows * ld) z += *reinterpret_cast<const f32x4_t*>(p);
    }
    const float at = lse[r], by = scale[r];
    const int t = target[r] - v0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float p = __builtin_amdgcn_exp2f((z[k] - at) * kLog2e);
      z[k] = c + k < cols ? (c + k == t ? p - 1.f : p) * by : 0.f;
    }
    store_mid<P>(g + r * g_ld + c, plane, z);
  }
}

// All of that for few rows, in one block: a wave a row.
template <typename I>
__global__ __launch_bounds__(1024) void k_loss_few(const float2* part, int strips, const I* targets,
                                                   int rows, int64_t ignore, int vocab,
                                                   const float* picked, float* loss, float* lse,
                                                   float* total, int mean) {
  __shared__ float each[kFewRows];
  __shared__ int counts[kFewRows];
  const int lane = threadIdx.x & 63, r = threadIdx.x >> 6;
  float value = 0.f;
  int count = 0;
  if (r < rows) {
    const int64_t t = (int64_t)targets[r];
    float m = -INFINITY, s = 0.f;
#pragma unroll 8
    for (int k = lane; k < strips; k += 64) {
      const float2 v = part[r * strips + k];
      const float top = fmaxf(m, v.x), ref = top == -INFINITY ? 0.f : top;
      s = s * __builtin_amdgcn_exp2f((m - ref) * kLog2e) +
          v.y * __builtin_amdgcn_exp2f((v.x - ref) * kLog2e);
      m = top;
    }
    float top = m;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
    const float ref = top == -INFINITY ? 0.f : top;
    s = lanes_sum<64>(s * __builtin_amdgcn_exp2f((m - ref) * kLog2e));
    const float ln = logf(s);
    const bool keep = t != ignore, there = t >= 0 && t < vocab;
    value = !keep ? 0.f : there ? ref - picked[r] + ln : NAN;
    count = keep;
    if (lane == 0) {
      lse[r] = keep ? ref + ln : 0.f;
      if (loss) loss[r] = value;
    }
  }
  if (!total) return;
  if (lane == 0) each[r] = value, counts[r] = count;
  __syncthreads();
  if (threadIdx.x == 0) {
    double sum = 0.0;
    int live = 0;
    for (int k = 0; k < rows; ++k) sum += each[k], live += counts[k];
    *total = (float)(mean && live ? sum / live : sum);
  }
}

// What the ignored rows hold, and the loss summed up (in double, in an order that
// the number of rows decides).  total: the sum, or the mean over the rows that
// count (0 where none does).
__global__ __launch_bounds__(1024) void k_loss_sum(const int32_t* pos, int rows,
                                                   const int32_t* count, float* loss, float* lse,
                                                   float* total, int mean) {
  __shared__ double sh[1024];
  double s = 0.0;
  for (int r = blockIdx.x * 1024 + threadIdx.x; r < rows; r += gridDim.x * 1024) {
    if (pos[r] < 0) loss[r] = lse[r] = 0.f;
    else s += loss[r];
  }
  if (!total) return;
  sh[threadIdx.x] = s;
  __syncthreads();
  for (int o = 512; o > 0; o >>= 1) {
    if ((int)threadIdx.x < o) sh[threadIdx.x] += sh[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    const int live = *count;
    *total = (float)(mean && live ? sh[0] / live : sh[0]);
  }
}

// Backward: what the epilogue needs of each row that counts, and the factor that
// they share (where no row counts there is nothing to multiply, whatever dloss is).
__global__ __launch_bounds__(256) void k_loss_rows(const int32_t* count, const int32_t* list,
                                                   const int32_t* target, const float* lse,
                                                   const float* dloss, int reduction, float* lse_at,
                                                   float* scale, float* by) {
  const int live = *count, i = blockIdx.x * 256 + threadIdx.x;
  if (i == 0)
    *by = live == 0 || reduction == SM_LOSS_ROWS ? 1.f
          : reduction == SM_LOSS_MEAN            ? *dloss / live
                                                 : *dloss;
  if (i >= live) return;
  const int r = list[i];
  lse_at[i] = lse[r];
  scale[i] = target[i] < 0 ? NAN : reduction == SM_LOSS_ROWS ? dloss[r] : 1.f;
}

namespace {

struct LossPlan {
  int planes, g_planes;
  int32_t dim_ld;                 // row length of operand copies
  bool copy_w, wide, thin;        // thin: the products with the table (sm_thin.h)
  int splits;                     // of the logits' k
  int64_t strips;
  // backward
  int64_t piece, g_ld;            // columns of a piece of the vocabulary, G's row length
  MmPlan both;                    // the products dX (job 0) and dW (job 1) of a piece
  // arrays
  int32_t *list, *target, *pos, *count;
  bf16_t *x, *w, *g;
  float *picked, *loss, *lse_at, *scale, *by, *dx, *dw;
  float* sums;                    // of the logits' splits
  float2* part;
  size_t bytes;
};

constexpr int64_t kTwoRows = 128, kTwoValues = 65536;    // up to which G has two planes
constexpr int64_t kPieceBytes = (int64_t)1 << 30;

// w_fits: the table is an operand as it lies
LossPlan loss_plan(int64_t rows, int64_t dim, int64_t vocab, int32_t dtype, bool w_fits,
                   bool backward, void* ws) {
  LossPlan p{};
  p.planes = dtype == SM_BF16 ? 1 : 3;
  p.dim_ld = (int32_t)operand_ld(dim);
  p.g_planes = p.planes == 3 ? 3 : rows <= kTwoRows || rows * dim <= kTwoValues ? 2 : 1;
  const int64_t most = std::max<int64_t>(256, kPieceBytes / (2 * p.g_planes * rows) / 256 * 256);
  const int64_t pieces = backward ? (vocab + most - 1) / most : 1;
  p.thin = thin_form(rows, vocab, dim, 1, dtype, backward) && pieces == 1;
  p.copy_w = !w_fits && !p.thin;
  Places at{static_cast<char*>(ws)};
  p.list = at.take<int32_t>(rows);
  p.target = at.take<int32_t>(rows);
  p.pos = at.take<int32_t>(rows);
  p.count = at.take<int32_t>(1);
  p.x = at.take<bf16_t>(p.planes * rows * p.dim_ld);
  if (p.copy_w) p.w = at.take<bf16_t>(p.planes * vocab * p.dim_ld);
  if (!backward && rows <= kFewRows) {
    Places few{static_cast<char*>(ws)};
    p.picked = few.take<float>(kFewRows);
    p.part = few.take<float2>(8192 * kFewRows);
    p.bytes = few.used;
    return p;
  }
  const auto logits_of = [&](int64_t cols) {
    if (p.thin) {
      p.splits = thin_splits(cols, rows, dim, 1);
      p.sums = at.take<float>(p.splits * rows * round_up(cols, 4));
      return;
    }
    const MmSize z{cols, rows, (p.planes == 1 ? 1 : 6) * ((dim + 63) / 64), true};
    const MmPlan plan = plan_products(&z, 1);
    p.wide = plan.wide;
    p.splits = plan.splits[0];
    if (p.splits > 1) p.sums = at.take<float>(p.splits * rows * round_up(cols, 4));
  };
  if (!backward) {
    logits_of(vocab);
    const int64_t strip = p.thin || p.splits > 1 ? kMidStrip : p.wide ? 128 : 64;
    p.strips = (vocab + strip - 1) / strip;
    p.loss = at.take<float>(rows);
    p.picked = at.take<float>(rows);
    p.part = at.take<float2>(p.strips * rows);
  } else {
    p.lse_at = at.take<float>(rows);
    p.scale = at.take<float>(rows);
    p.by = at.take<float>(1);
    p.piece = std::min(round_up((vocab + pieces - 1) / pieces, 256), round_up(vocab, 8));
    p.g_ld = operand_ld(p.piece);
    logits_of(std::min(p.piece, vocab));
    p.g = at.take<bf16_t>(p.g_planes * rows * p.g_ld);
    const int segs = p.planes == 1 ? p.g_planes : 6;
    const MmSize sizes[2] = {{dim, rows, segs * ((p.piece + 63) / 64), true},
                             {dim, p.piece, segs * ((rows + 63) / 64), true}};
    if (p.thin) {
      p.both = plan_products(sizes + 1, 1);
      p.both.splits[1] = p.both.splits[0];
      p.both.splits[0] = thin_splits(dim, rows, vocab, 1);
    } else {
      p.both = plan_products(sizes, 2);
    }
    // (dX is summed up over pieces and has its rows to be placed: always in parts)
    p.dx = at.take<float>(p.both.splits[0] * rows * round_up(dim, 4));
    if (p.both.splits[1] > 1) p.dw = at.take<float>(p.both.splits[1] * p.piece * round_up(dim, 4));
  }
  p.bytes = at.used;
  return p;
}

template <typename A>
hipError_t gather(const LossPlan& p, const A& a, hipStream_t s) {
  const auto list = [&](auto* t) {
    hipLaunchKernelGGL(k_loss_list, dim3(1), dim3(1024), 0, s, t, (int)a.rows, a.ignore, p.list,
                       p.target, p.pos, p.count, (int)a.vocab);
  };
  if (a.target_bits == 64) list(static_cast<const int64_t*>(a.targets));
  else list(static_cast<const int32_t*>(a.targets));
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  PlanesJobs c{};
  c.job[c.jobs++] = {a.X, a.x_stride, a.rows, (int)a.dim, p.dim_ld, p.list, p.count, p.x};
  if (p.copy_w)
    c.job[c.jobs++] = {a.W, a.dim, a.vocab, (int)a.dim, p.dim_ld, nullptr, nullptr, p.w};
  return launch_planes(c, a.dtype, s);
}

// The logits of rows [v0, v0 + cols) of the table.
MmArgs logits(const LossPlan& p, const void* W, int64_t rows, int64_t dim, int64_t vocab,
              int64_t v0, int64_t cols) {
  MmArgs m{};
  m.jobs = 1;
  MmJob& j = m.job[0];
  j.n_rows = p.count;
  j.lda = p.copy_w ? p.dim_ld : dim;
  j.a = (p.copy_w ? (const char*)p.w : (const char*)W) + v0 * j.lda * 2;
  j.b = (const char*)p.x;
  j.ldb = p.dim_ld;
  j.m = (int)cols;
  j.n = (int)rows;
  j.k = (int)dim;
  j.splits = p.splits;
  set_planes(j, p.planes, p.planes, vocab * p.dim_ld * 2, rows * p.dim_ld * 2);
  return m;
}

// Their sums of splits, for a launch of its own.
template <typename A>
hipError_t logit_sums(const LossPlan& p, MmArgs& m, const A& a, hipStream_t s) {
  if (p.thin) {
    // (rows past the count hold whatever there was, and nothing reads their sums)
    const ThinArgs t{{(const float*)a.W, nullptr}, {p.x, nullptr}, {p.sums, nullptr}, a.dim,
                     p.dim_ld, a.rows * p.dim_ld, (int)a.vocab, (int)a.rows, (int)a.dim, p.splits,
                     1, a.vocab * a.dim * 4 > kCacheBytes};
    return launch_thin<false>(t, s);
  }
  EpiStore::Args e{};
  e.out[0] = sums_out(p.sums, m.job[0].m, m.job[0].n);
  return run_mm<false, false, false, EpiStore>(m, e, p.wide, s);
}

template <int P>
hipError_t loss_grad_piece(const LossPlan& p, const LossGradArgs& a, int64_t v0, hipStream_t s) {
  const int64_t cols = std::min(p.piece, a.vocab - v0), plane = a.rows * p.g_ld;
  MmArgs m = logits(p, a.W, a.rows, a.dim, a.vocab, v0, cols);
  const char* w = m.job[0].a;
  const int64_t ldw = m.job[0].lda;
  if (p.thin || p.splits > 1) {
    SM_TRY(logit_sums(p, m, a, s));
    const int64_t work = a.rows * (round_up(cols, 8) / 4);
    hipLaunchKernelGGL((k_loss_mid_grad<P>),
                       dim3((unsigned)std::min<int64_t>((work + 255) / 256, 1 << 16)), dim3(256), 0,
                       s, p.sums, p.splits, p.count, (int)a.rows, (int)cols, p.target, (int)v0,
                       p.lse_at, p.scale, p.g, p.g_ld, plane);
    SM_TRY(hipGetLastError());
  } else {
    const typename EpiGrad<P>::Args eg{p.g, p.g_ld, plane, (int)v0, p.target, p.lse_at, p.scale};
    SM_TRY((run_mm<false, false, false, EpiGrad<P>>(m, eg, p.wide, s)));
  }
  MmStores out;
  if (a.dX && p.thin) {
    const ThinArgs t{{(const float*)a.W, nullptr}, {p.g, nullptr}, {p.dx, nullptr}, a.dim, p.g_ld,
                     plane, (int)a.dim, (int)a.rows, (int)a.vocab, p.both.splits[0], 1,
                     a.vocab * a.dim * 4 > kCacheBytes};
    SM_TRY(launch_thin<true>(t, s));
  } else if (a.dX) {
    MmJob j{};
    j.n_rows = p.count;
    j.a = w;
    j.lda = ldw;
    j.b = (const char*)p.g;
    j.ldb = p.g_ld;
    j.m = (int)a.dim;
    j.n = (int)a.rows;
    j.k = (int)cols;
    set_planes(j, p.planes, P, a.vocab * p.dim_ld * 2, plane * 2);
    const int64_t ld = round_up(a.dim, 4);
    out.add(j, false, nullptr, SM_F32, 0, p.dx, 1);
    out.a.job[0].splits = p.both.splits[0];
    out.e.out[0] = {p.dx, ld, a.rows * ld, SM_F32, v0 > 0, nullptr};
  }
  if (a.dW) {
    MmJob j{};
    j.k_rows = p.count;
    j.a = (const char*)p.x;
    j.lda = p.dim_ld;
    j.b = (const char*)p.g;
    j.ldb = p.g_ld;
    j.m = (int)a.dim;
    j.n = (int)cols;
    j.k = (int)a.rows;
    set_planes(j, p.planes, P, a.rows * p.dim_ld * 2, plane * 2);
    const int64_t size = a.dw_dtype == SM_F32 ? 4 : 2;
    out.add(j, true, static_cast<char*>(a.dW) + v0 * a.dim * size, a.dw_dtype, a.accumulate, p.dw,
            p.both.splits[1], p.by);
  }
  return out.run(p.both.wide, s);
}

}  // namespace

size_t loss_workspace(int64_t rows, int64_t dim, int64_t vocab, int32_t dtype, bool backward) {
  if (rows == 0) return 0;
  // room for a table that has to be copied
  return loss_plan(rows, dim, vocab, dtype, false, backward, nullptr).bytes;
}

template <typename T>
static hipError_t loss_few(const LossArgs& a, const LossPlan& p, hipStream_t s) {
  const int strips = few_strips<T>(a.vocab, a.dim);
  SM_TRY((launch_few<T, T, 1, FewLse<T>>((const T*)a.W, nullptr, a.dim, a.vocab, (const T*)a.X,
                                         a.x_stride, a.rows, a.dim,
                                         {p.part, strips, a.targets, a.target_bits, p.picked}, s)));
  float* loss = a.reduction == SM_LOSS_ROWS ? a.loss : nullptr;
  float* total = a.reduction == SM_LOSS_ROWS ? nullptr : a.loss;
  const auto join = [&](auto* t) {
    hipLaunchKernelGGL((k_loss_few<std::remove_const_t<std::remove_pointer_t<decltype(t)>>>),
                       dim3(1), dim3(1024), 0, s, p.part, strips, t, (int)a.rows, a.ignore,
                       (int)a.vocab, p.picked, loss, a.lse, total,
                       (int)(a.reduction == SM_LOSS_MEAN));
  };
  if (a.target_bits == 64) join(static_cast<const int64_t*>(a.targets));
  else join(static_cast<const int32_t*>(a.targets));
  return hipGetLastError();
}

hipError_t launch_loss(const LossArgs& a, hipStream_t s) {
  if (a.rows == 0) return launch_zero(a.loss, SM_F32, 1, s);
  const LossPlan p = loss_plan(a.rows, a.dim, a.vocab, a.dtype,
                               operand_fits(a.W, a.dtype, a.dim, a.dim), false, a.ws);
  if (a.rows <= kFewRows)
    return a.dtype == SM_BF16 ? loss_few<bf16_t>(a, p, s) : loss_few<float>(a, p, s);
  if (hipError_t e = gather(p, a, s); e != hipSuccess) return e;
  MmArgs m = logits(p, a.W, a.rows, a.dim, a.vocab, 0, a.vocab);
  float* loss = a.reduction == SM_LOSS_ROWS ? a.loss : p.loss;
  const EpiLse::Args e{p.part, a.rows, p.target, p.picked};
  if (p.thin || p.splits > 1) {
    SM_TRY(logit_sums(p, m, a, s));
    hipLaunchKernelGGL(k_loss_mid, dim3((unsigned)((a.rows * p.strips + 3) / 4)), dim3(256), 0, s,
                       p.sums, p.splits, p.count, (int)a.rows, (int)a.vocab, (int)p.strips, e);
    SM_TRY(hipGetLastError());
  } else {
    SM_TRY((run_mm<false, false, false, EpiLse>(m, e, p.wide, s)));
  }
  hipLaunchKernelGGL(k_loss_join, dim3((unsigned)((a.rows + 15) / 16)), dim3(1024), 0, s, p.part,
                     a.rows, (int)p.strips, p.count, p.list, p.target, p.picked, loss, a.lse);
  SM_TRY(hipGetLastError());
  hipLaunchKernelGGL(k_loss_sum, dim3(1), dim3(1024), 0, s, p.pos, (int)a.rows, p.count, loss,
                     a.lse, a.reduction == SM_LOSS_ROWS ? nullptr : a.loss,
                     (int)(a.reduction == SM_LOSS_MEAN));
  return hipGetLastError();
}

hipError_t launch_loss_grad(const LossGradArgs& a, hipStream_t s) {
  if (a.rows == 0)        // a sum of nothing
    return a.dW && !a.accumulate ? launch_zero(a.dW, a.dw_dtype, a.vocab * a.dim, s) : hipSuccess;
  const LossPlan p = loss_plan(a.rows, a.dim, a.vocab, a.dtype,
                               operand_fits(a.W, a.dtype, a.dim, a.dim), true, a.ws);
  if (hipError_t e = gather(p, a, s); e != hipSuccess) return e;
  hipLaunchKernelGGL(k_loss_rows, dim3((unsigned)((a.rows + 255) / 256)), dim3(256), 0, s, p.count,
                     p.list, p.target, a.lse, a.dloss, (int)a.reduction, p.lse_at, p.scale, p.by);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  for (int64_t v0 = 0; v0 < a.vocab; v0 += p.piece) {
    const hipError_t e = p.g_planes == 1   ? loss_grad_piece<1>(p, a, v0, s)
                         : p.g_planes == 2 ? loss_grad_piece<2>(p, a, v0, s)
                                           : loss_grad_piece<3>(p, a, v0, s);
    if (e != hipSuccess) return e;
  }
  if (!a.dX) return hipSuccess;
  const int64_t ld = round_up(a.dim, 4);
  JoinJobs j{};
  j.job[j.jobs++] = {p.dx, a.rows * ld, ld, p.both.splits[0], p.pos, a.rows, (int)a.dim, a.dtype, 0,
                     a.dX, a.dim, p.by};
  return launch_join(j, s);
}

}  // namespace sm
