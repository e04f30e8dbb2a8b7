// Gated feed-forward block (signmuon_layers.h), forward and backward:
//   y = (act(x Wg^T) * (x Wu^T)) Wd^T.
//
// Forward, two products: the rows of Wg and Wu alternate in groups of 16 in the
// first one's tiles, so that a lane holds a gate and its up value, and the
// epilogue writes the activations alone (and, for training, the two
// pre-activations in float32: their errors reach every gradient, and rounded to
// bfloat16 they would double it).  Backward, three launches: dh = dy Wd with the
// activation's derivative in its epilogue, which writes dg, du and h; dx = dg Wg
// + du Wu, one sum over both; and the three weight gradients.  What is between
// the products is rounded to the operands' type: for bfloat16 half a step of 2^-8
// a value, as much as the rounding of the results.  Together they leave a result's
// error at sqrt(2) of its own rounding where errors average; where it comes from few
// values, or is few values, that can be twice as much: there they have two
// bfloat16 planes.
//
// Up to 16 rows the products are bound by reading the weights once (sm_few.h): one
// row, 4096 x 16384, 47 + 26 us.  4096 rows of it: 1037 us for gate and up with
// their epilogue (1060 TFLOP/s, and 0.7 GB written), 465 for the last product (1180);
// the chip's power bounds both.  Backward, 12288 rows of 768 x 2048: 163 us
// for dh with its epilogue, which reads 201 MB of pre and writes 151 MB beside 39
// GFLOP and runs beside no product, and 270 for the rest in one launch (193 GFLOP in
// 864 unsplit tiles of 128 x 128).
#include "sm_few.h"
#include "sm_thin.h"
#include "sm_layers.h"
#include "sm_mm_ops.h"

namespace sm {

constexpr float kLog2e = 1.44269504088896341f;

// Act 0: silu, x / (1 + exp(-x)); 1: gelu, x Phi(x).
__device__ __forceinline__ float sigmoid(float g) {
  return 1.0f / (1.0f + __builtin_amdgcn_exp2f(-kLog2e * g));
}
__device__ __forceinline__ float phi(float g) { return 0.5f * (1.0f + erff(g * 0.70710678118f)); }
template <int ACT>
__device__ __forceinline__ float act(float g) {
  return g * (ACT == 0 ? sigmoid(g) : phi(g));
}
// the activation and its derivative
template <int ACT>
__device__ __forceinline__ void act_slope(float g, float& a, float& slope) {
  if constexpr (ACT == 0) {
    const float s = sigmoid(g);
    a = g * s;
    slope = s * (1.0f + g * (1.0f - s));
  } else {
    const float p = phi(g);
    a = g * p;
    slope = p + g * (0.39894228040f * __builtin_amdgcn_exp2f(-0.5f * kLog2e * g * g));
  }
}

// h = act(gate) * up of a paired product, to planes of [rows][ld]; pre: gate and
// up, [rows][2 hidden], or NULL.
template <int P, int ACT>
struct EpiGate {
  struct Args {
    bf16_t* h;
    int64_t ld, plane;
    float* pre;
  };
  template <int TI, int TJ>
  static __device__ __forceinline__ void run(const Args& e, const MmPlace& at,
                                             const f32x4_t (&acc)[TI][TJ]) {
    constexpr int F = 8 * TI;                        // features of a wave
    const int cols = at.m - at.m0;
    const int cols8 = ((at.m + 7) & ~7) - at.m0;     // zeros up to a whole piece of 16 bytes
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      // (features past the last one are products of zeros)
      f32x4_t g[TI / 2], u[TI / 2], h[TI / 2];
#pragma unroll
      for (int i = 0; i < TI / 2; ++i) {
        g[i] = acc[2 * i][j];
        u[i] = acc[2 * i + 1][j];
#pragma unroll
        for (int k = 0; k < 4; ++k) h[i][k] = act<ACT>(g[i][k]) * u[i][k];
      }
      const int n = at.n0 + 16 * j;
      put_planes<P, F>(at, h, e.h + (int64_t)n * e.ld + at.m0, e.plane, e.ld, at.n - n, cols8);
      if (e.pre) {
        const MmRows<float, F> rows{at.lds, at.lane};
        float* p = e.pre + (int64_t)n * 2 * at.m + at.m0;
#pragma unroll
        for (int i = 0; i < TI / 2; ++i) rows.put(0, i, g[i]), rows.put(1, i, u[i]);
        rows.flush(0, p, 2 * at.m, at.n - n, cols);
        rows.flush(1, p + at.m, 2 * at.m, at.n - n, cols);
      }
    }
  }
};

// From dh and the pre-activations: dg = dh up act'(gate), du = dh act(gate),
// h = act(gate) up, planes of [rows][ld].
template <int P, int ACT>
struct EpiGateGrad {
  struct Args {
    bf16_t *dg, *du, *h;
    int64_t ld, plane;
    const float* pre;
  };
  template <int TI, int TJ>
  static __device__ __forceinline__ void run(const Args& e, const MmPlace& at,
                                             const f32x4_t (&acc)[TI][TJ]) {
    constexpr int F = 16 * TI;
    const int mc = at.m0 + 4 * (at.lane >> 4), nc = at.n0 + (at.lane & 15);
    const int cols8 = ((at.m + 7) & ~7) - at.m0;     // zeros up to a whole piece of 16 bytes
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const int n = nc + 16 * j;
      const float* p = e.pre + (int64_t)(n < at.n ? n : at.n - 1) * 2 * at.m;
      const int n0 = at.n0 + 16 * j;
      const int64_t o = (int64_t)n0 * e.ld + at.m0;
      const auto values = [&](int i, f32x4_t& dg, f32x4_t& du, f32x4_t& h) SM_INLINE {
        const int f = mc + 16 * i;
        float g[4], u[4];
        if (f + 4 <= at.m) {
          Piece<float, 4> pg, pu;
          pg.load(p + f);
          pu.load(p + at.m + f);
#pragma unroll
          for (int k = 0; k < 4; ++k) g[k] = pg[k], u[k] = pu[k];
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            g[k] = f + k < at.m ? p[f + k] : 0.f;
            u[k] = f + k < at.m ? p[at.m + f + k] : 0.f;
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float dh = f + k < at.m ? acc[i][j][k] : 0.f;
          float a, slope;
          act_slope<ACT>(g[k], a, slope);
          dg[k] = dh * u[k] * slope;
          du[k] = dh * a;
          h[k] = a * u[k];
        }
      };
      if constexpr (P == 1) {
        const MmRows<bf16_t, F> rows{at.lds, at.lane};
#pragma unroll
        for (int i = 0; i < TI; ++i) {
          f32x4_t dg, du, h;
          values(i, dg, du, h);
          rows.put(0, i, dg);
          rows.put(1, i, du);
          rows.put(2, i, h);
        }
        rows.flush(0, e.dg + o, e.ld, at.n - n0, cols8);
        rows.flush(1, e.du + o, e.ld, at.n - n0, cols8);
        rows.flush(2, e.h + o, e.ld, at.n - n0, cols8);
      } else {
        // one after the other: nine planes do not fit the wave's LDS, nor the
        // values of all three its registers
        const auto one = [&](auto which, bf16_t* dst) SM_INLINE {
          f32x4_t v[TI];
#pragma unroll
          for (int i = 0; i < TI; ++i) {
            f32x4_t t[3];
            values(i, t[0], t[1], t[2]);
            v[i] = t[decltype(which)::value];
          }
          put_planes<P, F>(at, v, dst + o, e.plane, e.ld, at.n - n0, cols8);
        };
        one(std::integral_constant<int, 0>(), e.dg);
        one(std::integral_constant<int, 1>(), e.du);
        one(std::integral_constant<int, 2>(), e.h);
      }
    }
  }
};

// The same for few rows: h of type H.
template <typename H, int ACT>
struct FewGate {
  struct Args {
    H* h;
    float* pre;
  };
  Args e;
  int lane, n;
  __device__ __forceinline__ FewGate(const Args& a, int l, int rows) : e(a), lane(l), n(rows) {}
  __device__ __forceinline__ void group(int m0, int m, const f32x4_t (&acc)[2]) {
    const int r = lane & 15, f = m0 + 4 * (lane >> 4);
    if (r >= n) return;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (f + k >= m) continue;
      put(e.h + (int64_t)r * m + f + k, act<ACT>(acc[0][k]) * acc[1][k]);
      if (e.pre) {
        e.pre[(int64_t)r * 2 * m + f + k] = acc[0][k];
        e.pre[(int64_t)r * 2 * m + m + f + k] = acc[1][k];
      }
    }
  }
  __device__ __forceinline__ void finish(int) {}
};
template <typename T>
struct FewStore {
  struct Args {
    T* y;
  };
  Args e;
  int lane, n;
  __device__ __forceinline__ FewStore(const Args& a, int l, int rows) : e(a), lane(l), n(rows) {}
  __device__ __forceinline__ void group(int m0, int m, const f32x4_t (&acc)[1]) {
    const int r = lane & 15, f = m0 + 4 * (lane >> 4);
    if (r >= n) return;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (f + k < m) put(e.y + (int64_t)r * m + f + k, acc[0][k]);
  }
  __device__ __forceinline__ void finish(int) {}
};

// What follows the first product where its k is split: the sums of the splits
// joined, and what the epilogues above do.  A thread has 4 features of a row.  333 x
// 2731 float32, backward, 10.6 us, bound by memory.
struct MidArgs {
  const float* sums[2];    // [split][rows][hidden rounded up to 4]: gate and up, or dh
  int32_t splits;
  int64_t rows;
  int32_t hidden, ld;
  int64_t plane;
  const float* pre;        // backward
  float* pre_out;          // forward, or null
  bf16_t* out[3];          // h; or dg, du, h
};
template <int P, int ACT, bool GRAD>
__global__ __launch_bounds__(256) void k_mid(MidArgs a) {
  const int hidden = a.hidden, hid4 = (hidden + 3) & ~3, per = ((hidden + 7) & ~7) / 4;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.rows * per;
       i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / per;
    const int f = (int)(i - r * per) * 4;
    f32x4_t s[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    if (f < hidden) {
#pragma unroll
      for (int w = 0; w < (GRAD ? 1 : 2); ++w) {
        const float* p = a.sums[w] + r * hid4 + f;
        for (int k = 0; k < a.splits; ++k, p += a.rows * hid4)
          s[w] += *reinterpret_cast<const f32x4_t*>(p);
      }
    }
    f32x4_t v[3];
    const int64_t pre = r * 2 * hidden + f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool in = f + k < hidden;
      if constexpr (GRAD) {
        const float g = in ? a.pre[pre + k] : 0.f, u = in ? a.pre[pre + hidden + k] : 0.f;
        const float dh = in ? s[0][k] : 0.f;
        float act_g, slope;
        act_slope<ACT>(g, act_g, slope);
        v[0][k] = dh * u * slope;
        v[1][k] = dh * act_g;
        v[2][k] = act_g * u;
      } else {
        const float g = in ? s[0][k] : 0.f, u = in ? s[1][k] : 0.f;
        v[0][k] = act<ACT>(g) * u;
        if (a.pre_out && in) a.pre_out[pre + k] = g, a.pre_out[pre + hidden + k] = u;
      }
    }
#pragma unroll
    for (int w = 0; w < (GRAD ? 3 : 1); ++w)
      store_mid<P>(a.out[w] + r * a.ld + f, a.plane, v[w]);
  }
}

namespace {

template <int P, int ACT, bool GRAD>
hipError_t launch_mid(const MidArgs& a, hipStream_t s) {
  const int64_t work = a.rows * (round_up(a.hidden, 8) / 4);
  hipLaunchKernelGGL((k_mid<P, ACT, GRAD>),
                     dim3((unsigned)std::min<int64_t>((work + 255) / 256, 1 << 16)), dim3(256), 0,
                     s, a);
  return hipGetLastError();
}
struct Operand {
  const char* p;
  int64_t ld, plane;       // elements; bytes from one plane to the next
};

struct FfnPlan {
  int planes, mid_planes;  // of the caller's operands; of what is between the products
  int64_t ld_d, ld_f;
  bf16_t *x, *dy, *wg, *wu, *wd, *h, *dg, *du;
  void* few_h;             // of few rows: bfloat16, or float32 for more planes
  MmPlan first, out;       // tiles of the first product; of the others (forward: y;
                           // backward: dx, dwg, dwu, dwd)
  float* sums[4];          // of their splits
  int thin[2];             // splits of the thin form's products
  bool split_first;        // the first product's k is split, and what follows it
  float* mid;              // takes a launch of its own: its sums
  size_t bytes;
};

constexpr int64_t kTwoPlanes = 4096;     // values below which there are two planes

FfnPlan ffn_plan(int64_t rows, int64_t dim, int64_t hidden, int32_t dtype, bool backward,
                 void* ws) {
  FfnPlan p{};
  p.planes = dtype == SM_BF16 ? 1 : 3;
  p.mid_planes = p.planes == 3 ? 3 : rows * std::min(dim, hidden) < kTwoPlanes ? 2 : 1;
  p.ld_d = operand_ld(dim);
  p.ld_f = operand_ld(hidden);
  Places at{static_cast<char*>(ws)};
  if (!backward && rows <= kFewRows) {
    p.few_h = at.take<float>(rows * hidden);    // (or half of it in bfloat16)
    p.bytes = at.used;
    return p;
  }
  const bool thin = thin_form(rows, dim, hidden, 3, dtype, backward);
  if (!backward && thin) {
    p.thin[0] = thin_splits(hidden, rows, dim, 2);
    p.thin[1] = thin_splits(dim, rows, hidden, 1);
    p.x = at.take<bf16_t>(3 * rows * p.ld_d);
    p.h = at.take<bf16_t>(3 * rows * p.ld_f);
    p.mid = at.take<float>(2 * p.thin[0] * rows * round_up(hidden, 4));
    p.sums[0] = at.take<float>(p.thin[1] * rows * round_up(dim, 4));
    p.bytes = at.used;
    return p;
  }
  const int64_t segs = p.planes == 1 ? 1 : 6, mid = p.planes == 1 ? p.mid_planes : 6;
  p.x = at.take<bf16_t>(p.planes * rows * p.ld_d);
  if (!thin) {
    p.wg = at.take<bf16_t>(p.planes * hidden * p.ld_d);
    p.wu = at.take<bf16_t>(p.planes * hidden * p.ld_d);
    p.wd = at.take<bf16_t>(p.planes * dim * p.ld_f);
  }
  p.h = at.take<bf16_t>(p.mid_planes * rows * p.ld_f);
  const auto first = [&](MmSize z, int jobs) {
    const MmSize both[2] = {z, z};
    p.first = plan_products(both, jobs);
    p.split_first = p.first.splits[0] > 1;
    if (p.split_first)
      p.mid = at.take<float>(jobs * p.first.splits[0] * rows * round_up(hidden, 4));
  };
  const auto slabs = [&](int64_t k) { return segs * ((k + 63) / 64); };
  const auto mids = [&](int64_t k) { return mid * ((k + 63) / 64); };
  const auto room = [&](const MmSize* z, int jobs) {
    p.out = plan_products(z, jobs);
    for (int i = 0; i < jobs; ++i)
      if (p.out.splits[i] > 1)
        p.sums[i] = at.take<float>(p.out.splits[i] * z[i].n * round_up(z[i].m, 4));
  };
  if (!backward) {
    const MmSize y{dim, rows, mids(hidden), true};
    first({hidden, rows, slabs(dim), true}, 2);
    room(&y, 1);
  } else {
    p.dy = at.take<bf16_t>(p.planes * rows * p.ld_d);
    p.dg = at.take<bf16_t>(p.mid_planes * rows * p.ld_f);
    p.du = at.take<bf16_t>(p.mid_planes * rows * p.ld_f);
    const MmSize o[4] = {{dim, rows, 2 * mids(hidden), true},
                         {dim, hidden, mids(rows), true},
                         {dim, hidden, mids(rows), true},
                         {hidden, dim, mids(rows), true}};
    if (thin) {
      p.thin[0] = thin_splits(hidden, rows, dim, 1);
      p.thin[1] = thin_splits(dim, rows, hidden, 2);
      p.mid = at.take<float>(p.thin[0] * rows * round_up(hidden, 4));
      p.sums[0] = at.take<float>(2 * p.thin[1] * rows * round_up(dim, 4));
      p.out = plan_products(o + 1, 3);
      for (int i = 3; i > 0; --i) {
        p.out.splits[i] = p.out.splits[i - 1];
        if (p.out.splits[i] > 1)
          p.sums[i] = at.take<float>(p.out.splits[i] * o[i].n * round_up(o[i].m, 4));
      }
    } else {
      first({hidden, rows, slabs(dim), true}, 1);
      room(o, 4);
    }
  }
  p.bytes = at.used;
  return p;
}

// An operand: where the caller's matrix lies, or a copy that `c` is to make.
Operand operand(PlanesJobs& c, const void* src, int32_t dtype, int64_t rows, int64_t cols,
                int64_t stride, bf16_t* copy, bool copied = false) {
  if (!copied && operand_fits(src, dtype, cols, stride))
    return {static_cast<const char*>(src), stride, 0};
  const int64_t ld = operand_ld(cols);
  c.job[c.jobs++] = {src, stride, rows, (int)cols, (int32_t)ld, nullptr, nullptr, copy};
  return {reinterpret_cast<const char*>(copy), ld, rows * ld * 2};
}

MmJob product(const Operand& a, const Operand& b, int64_t m, int64_t n, int64_t k, int a_planes,
              int b_planes) {
  MmJob j{};
  j.a = a.p;
  j.b = b.p;
  j.lda = a.ld;
  j.ldb = b.ld;
  j.m = (int)m;
  j.n = (int)n;
  j.k = (int)k;
  j.splits = 1;
  set_planes(j, a_planes, b_planes, a.plane, b.plane);
  return j;
}

template <typename T, typename H, int ACT>
hipError_t ffn_few(const FfnArgs& a, const FfnPlan& p, hipStream_t s) {
  SM_TRY((launch_few<T, T, 2, FewGate<H, ACT>>((const T*)a.Wg, (const T*)a.Wu, a.dim, a.hidden,
                                               (const T*)a.X, a.x_stride, a.rows, a.dim,
                                               {(H*)p.few_h, a.pre}, s)));
  return launch_few<T, H, 1, FewStore<T>>((const T*)a.Wd, nullptr, a.hidden, a.dim,
                                          (const H*)p.few_h, a.hidden, a.rows, a.hidden,
                                          {(T*)a.Y}, s);
}

// float32 and few rows more (sm_thin.h).
template <int ACT>
hipError_t ffn_thin(const FfnArgs& a, const FfnPlan& p, hipStream_t s) {
  PlanesJobs c{};
  c.job[c.jobs++] = {a.X, a.x_stride, a.rows, (int)a.dim, (int)p.ld_d, nullptr, nullptr, p.x};
  SM_TRY(launch_planes(c, a.dtype, s));
  const bool once = 12 * a.dim * a.hidden > kCacheBytes;
  float* up = p.mid + p.thin[0] * a.rows * round_up(a.hidden, 4);
  const ThinArgs first{{(const float*)a.Wg, (const float*)a.Wu}, {p.x, p.x}, {p.mid, up}, a.dim,
                       p.ld_d, a.rows * p.ld_d, (int)a.hidden, (int)a.rows, (int)a.dim, p.thin[0],
                       2, once};
  SM_TRY(launch_thin<false>(first, s));
  const int64_t plane = a.rows * p.ld_f;
  const MidArgs g{{p.mid, up}, p.thin[0], a.rows, (int)a.hidden, (int)p.ld_f, plane, nullptr, a.pre,
                  {p.h, nullptr, nullptr}};
  SM_TRY((launch_mid<3, ACT, false>(g, s)));
  const ThinArgs out{{(const float*)a.Wd, nullptr}, {p.h, nullptr}, {p.sums[0], nullptr}, a.hidden,
                     p.ld_f, plane, (int)a.dim, (int)a.rows, (int)a.hidden, p.thin[1], 1, once};
  SM_TRY(launch_thin<false>(out, s));
  const int64_t ld = round_up(a.dim, 4);
  JoinJobs j{};
  j.job[j.jobs++] = {p.sums[0], a.rows * ld, ld, p.thin[1], nullptr, a.rows, (int)a.dim, a.dtype, 0,
                     a.Y, a.dim, nullptr};
  return launch_join(j, s);
}

template <int P, int MP, int ACT>
hipError_t ffn(const FfnArgs& a, const FfnPlan& p, hipStream_t s) {
  // (Wg and Wu lie where they are, or both are copied: they share a row length)
  const bool copied = !operand_fits(a.Wg, a.dtype, a.dim, a.dim) ||
                      !operand_fits(a.Wu, a.dtype, a.dim, a.dim);
  PlanesJobs c{};
  const Operand x = operand(c, a.X, a.dtype, a.rows, a.dim, a.x_stride, p.x);
  const Operand wg = operand(c, a.Wg, a.dtype, a.hidden, a.dim, a.dim, p.wg, copied);
  const Operand wu = operand(c, a.Wu, a.dtype, a.hidden, a.dim, a.dim, p.wu, copied);
  const Operand wd = operand(c, a.Wd, a.dtype, a.dim, a.hidden, a.hidden, p.wd);
  SM_TRY(launch_planes(c, a.dtype, s));
  const int64_t plane = a.rows * p.ld_f;
  const Operand h{(const char*)p.h, p.ld_f, plane * 2};
  if (p.split_first) {
    MmStores z;
    float* sums[2] = {p.mid, p.mid + p.first.splits[0] * a.rows * round_up(a.hidden, 4)};
    for (int i = 0; i < 2; ++i) {
      z.add(product(i ? wu : wg, x, a.hidden, a.rows, a.dim, P, P), false, nullptr, SM_F32, 0,
            sums[i], p.first.splits[0]);
      z.e.out[i] = sums_out(sums[i], a.hidden, a.rows);
    }
    SM_TRY((run_mm<false, false, false, EpiStore>(z.a, z.e, p.first.wide, s)));
    const MidArgs g{{sums[0], sums[1]}, p.first.splits[0], a.rows, (int)a.hidden, (int)p.ld_f,
                    plane, nullptr, a.pre, {p.h, nullptr, nullptr}};
    SM_TRY((launch_mid<MP, ACT, false>(g, s)));
  } else {
    MmArgs m{};
    m.jobs = 1;
    m.job[0] = product(wg, x, a.hidden, a.rows, a.dim, P, P);
    m.job[0].a2 = wu.p;
    SM_TRY((run_mm<false, false, true, EpiGate<MP, ACT>>(m, {p.h, p.ld_f, plane, a.pre},
                                                         p.first.wide, s)));
  }
  MmStores out;
  out.add(product(wd, h, a.dim, a.rows, a.hidden, P, MP), false, a.Y, a.dtype, 0, p.sums[0],
          p.out.splits[0]);
  SM_TRY((run_mm<false, false, false, EpiStore>(out.a, out.e, p.out.wide, s)));
  return out.joins(s);
}

template <int P, int MP, int ACT>
hipError_t ffn_grad(const FfnGradArgs& a, const FfnPlan& p, hipStream_t s) {
  const bool thin = thin_form(a.rows, a.dim, a.hidden, 3, a.dtype, true);
  const bool copied = !operand_fits(a.Wg, a.dtype, a.dim, a.dim) ||
                      !operand_fits(a.Wu, a.dtype, a.dim, a.dim);
  PlanesJobs c{};
  const Operand dy = operand(c, a.dY, a.dtype, a.rows, a.dim, a.dy_stride, p.dy);
  Operand x{}, wd{}, wg{}, wu{};
  if (!thin) wd = operand(c, a.Wd, a.dtype, a.dim, a.hidden, a.hidden, p.wd);
  if (a.dX && !thin) {
    wg = operand(c, a.Wg, a.dtype, a.hidden, a.dim, a.dim, p.wg, copied);
    wu = operand(c, a.Wu, a.dtype, a.hidden, a.dim, a.dim, p.wu, copied);
  }
  if (a.dWg || a.dWu) x = operand(c, a.X, a.dtype, a.rows, a.dim, a.x_stride, p.x);
  SM_TRY(launch_planes(c, a.dtype, s));
  const int64_t plane = a.rows * p.ld_f;
  const MmJob first = product(wd, dy, a.hidden, a.rows, a.dim, P, P);
  const bool once = 12 * a.dim * a.hidden > kCacheBytes;
  if (thin) {
    const ThinArgs t{{(const float*)a.Wd, nullptr}, {p.dy, nullptr}, {p.mid, nullptr}, a.hidden,
                     p.ld_d, a.rows * p.ld_d, (int)a.hidden, (int)a.rows, (int)a.dim, p.thin[0], 1,
                     once};
    SM_TRY(launch_thin<true>(t, s));
    const MidArgs g{{p.mid, nullptr}, p.thin[0], a.rows, (int)a.hidden, (int)p.ld_f, plane, a.pre,
                    nullptr, {p.dg, p.du, p.h}};
    SM_TRY((launch_mid<MP, ACT, true>(g, s)));
  } else if (p.split_first) {
    MmStores z;
    z.add(first, false, nullptr, SM_F32, 0, p.mid, p.first.splits[0]);
    z.e.out[0] = sums_out(p.mid, a.hidden, a.rows);
    SM_TRY((run_mm<true, false, false, EpiStore>(z.a, z.e, p.first.wide, s)));
    const MidArgs g{{p.mid, nullptr}, p.first.splits[0], a.rows, (int)a.hidden, (int)p.ld_f,
                    plane, a.pre, nullptr, {p.dg, p.du, p.h}};
    SM_TRY((launch_mid<MP, ACT, true>(g, s)));
  } else {
    MmArgs m{};
    m.jobs = 1;
    m.job[0] = first;
    SM_TRY((run_mm<true, false, false, EpiGateGrad<MP, ACT>>(
        m, {p.dg, p.du, p.h, p.ld_f, plane, a.pre}, p.first.wide, s)));
  }
  const Operand dg{(const char*)p.dg, p.ld_f, plane * 2};
  const Operand du{(const char*)p.du, p.ld_f, plane * 2};
  const Operand h{(const char*)p.h, p.ld_f, plane * 2};
  MmStores out;
  if (a.dX && thin) {
    const int64_t ld = round_up(a.dim, 4), step = a.rows * ld;
    const ThinArgs t{{(const float*)a.Wg, (const float*)a.Wu}, {p.dg, p.du},
                     {p.sums[0], p.sums[0] + p.thin[1] * step}, a.dim, p.ld_f, plane, (int)a.dim,
                     (int)a.rows, (int)a.hidden, p.thin[1], 2, once};
    SM_TRY(launch_thin<true>(t, s));
    JoinJobs j{};
    j.job[j.jobs++] = {p.sums[0], step, ld, 2 * p.thin[1], nullptr, a.rows, (int)a.dim, a.dtype, 0,
                       a.dX, a.dim, nullptr};
    SM_TRY(launch_join(j, s));
  } else if (a.dX) {
    MmJob j = product(wg, dg, a.dim, a.rows, a.hidden, P, MP);
    j.parts = 2;
    j.a_part = wu.p - wg.p;
    j.b_part = du.p - dg.p;
    out.add(j, false, a.dX, a.dtype, 0, p.sums[0], p.out.splits[0]);
  }
  const auto add = [&](int i, const Operand& A, const Operand& B, void* dst, int64_t mm,
                       int64_t nn) {
    if (dst)
      out.add(product(A, B, mm, nn, a.rows, i == 3 ? MP : P, i == 3 ? P : MP), true, dst,
              a.dw_dtype, a.accumulate, p.sums[i], p.out.splits[i]);
  };
  add(1, x, dg, a.dWg, a.dim, a.hidden);
  add(2, x, du, a.dWu, a.dim, a.hidden);
  add(3, h, dy, a.dWd, a.hidden, a.dim);
  return out.run(p.out.wide, s);
}

}  // namespace

size_t ffn_workspace(int64_t rows, int64_t dim, int64_t hidden, int32_t dtype, bool backward) {
  return rows == 0 ? 0 : ffn_plan(rows, dim, hidden, dtype, backward, nullptr).bytes;
}

hipError_t launch_ffn(const FfnArgs& a, hipStream_t s) {
  const FfnPlan p = ffn_plan(a.rows, a.dim, a.hidden, a.dtype, false, a.ws);
  const auto go = [&](auto act) {
    constexpr int ACT = decltype(act)::value;
    if (a.rows <= kFewRows)
      return p.mid_planes == 1   ? ffn_few<bf16_t, bf16_t, ACT>(a, p, s)
             : p.mid_planes == 2 ? ffn_few<bf16_t, float, ACT>(a, p, s)
                                 : ffn_few<float, float, ACT>(a, p, s);
    if (thin_form(a.rows, a.dim, a.hidden, 3, a.dtype, false)) return ffn_thin<ACT>(a, p, s);
    return p.mid_planes == 1   ? ffn<1, 1, ACT>(a, p, s)
           : p.mid_planes == 2 ? ffn<1, 2, ACT>(a, p, s)
                               : ffn<3, 3, ACT>(a, p, s);
  };
  return a.act == SM_ACT_SILU ? go(std::integral_constant<int, 0>())
                              : go(std::integral_constant<int, 1>());
}

hipError_t launch_ffn_grad(const FfnGradArgs& a, hipStream_t s) {
  if (a.rows == 0) {           // sums of nothing
    if (a.accumulate) return hipSuccess;
    for (void* p : {a.dWg, a.dWu, a.dWd})
      if (p) SM_TRY(launch_zero(p, a.dw_dtype, a.dim * a.hidden, s));
    return hipSuccess;
  }
  const FfnPlan p = ffn_plan(a.rows, a.dim, a.hidden, a.dtype, true, a.ws);
  const auto go = [&](auto act) {
    constexpr int ACT = decltype(act)::value;
    return p.mid_planes == 1   ? ffn_grad<1, 1, ACT>(a, p, s)
           : p.mid_planes == 2 ? ffn_grad<1, 2, ACT>(a, p, s)
                               : ffn_grad<3, 3, ACT>(a, p, s);
  };
  return a.act == SM_ACT_SILU ? go(std::integral_constant<int, 0>())
                              : go(std::integral_constant<int, 1>());
}

}  // namespace sm
