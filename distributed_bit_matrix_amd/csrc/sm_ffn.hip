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
// the products is rounded to the operands' type: for bfloat16 half a step of
// 2^-8 a value, as much as the rounding of the results.
//
// Up to 16 rows the products are bound by reading the weights once (sm_few.h).
#include "sm_few.h"
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
    const int mc = at.m0 + 4 * (at.lane >> 4), nc = at.n0 + (at.lane & 15);
    const int m_end = (at.m + 7) & ~7;     // zeros up to a whole piece of 16 bytes
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const int n = nc + 16 * j;
      if (n >= at.n) continue;
#pragma unroll
      for (int i = 0; i < TI; i += 2) {
        const int f = mc + 8 * i;
        if (f >= m_end) continue;
        float v[4], g[4], u[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          g[k] = acc[i][j][k];
          u[k] = acc[i + 1][j][k];
          v[k] = f + k < at.m ? act<ACT>(g[k]) * u[k] : 0.f;
        }
        store_planes<P>(e.h + (int64_t)n * e.ld + f, e.plane, v);
        if (e.pre) {
          float* p = e.pre + (int64_t)n * 2 * at.m + f;
          if (f + 4 <= at.m) {
            store_vec<4>(p, g);
            store_vec<4>(p + at.m, u);
          } else {
            for (int k = 0; k < at.m - f; ++k) p[k] = g[k], p[at.m + k] = u[k];
          }
        }
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
    const int mc = at.m0 + 4 * (at.lane >> 4), nc = at.n0 + (at.lane & 15);
    const int m_end = (at.m + 7) & ~7;
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const int n = nc + 16 * j;
      if (n >= at.n) continue;
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        const int f = mc + 16 * i;
        if (f >= m_end) continue;
        const float* p = e.pre + (int64_t)n * 2 * at.m + f;
        float dg[4], du[4], h[4], g[4], u[4];
        if (f + 4 <= at.m) {
          Piece<float, 4> pg, pu;
          pg.load(p);
          pu.load(p + at.m);
#pragma unroll
          for (int k = 0; k < 4; ++k) g[k] = pg[k], u[k] = pu[k];
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            g[k] = f + k < at.m ? p[k] : 0.f;
            u[k] = f + k < at.m ? p[at.m + k] : 0.f;
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
        const int64_t o = (int64_t)n * e.ld + f;
        store_planes<P>(e.dg + o, e.plane, dg);
        store_planes<P>(e.du + o, e.plane, du);
        store_planes<P>(e.h + o, e.plane, h);
      }
    }
  }
};

// The same for few rows: h in the weights' type.
template <typename T, int ACT>
struct FewGate {
  struct Args {
    T* h;
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

namespace {

// An operand: the caller's matrix where it fits, else a copy.
struct Operand {
  const char* p;
  int64_t ld, plane;       // elements; bytes from one plane to the next
  bf16_t* copy;
};

struct FfnPlan {
  int planes;
  int64_t ld_d, ld_f;
  bf16_t *x, *dy, *wg, *wu, *wd, *h, *dg, *du;
  void* few_h;
  float* part[4];          // sums of splits: dx, dwg, dwu, dwd (forward: y first)
  int splits[4];
  bool wide[4];
  size_t bytes;
};

// Splits and tiles of a product, and room for its sums.
void plan_product(FfnPlan& p, Places& at, int i, int64_t m, int64_t n, int64_t k) {
  p.wide[i] = wide_tiles(m, n);
  p.splits[i] = k_splits(m, n, (k + 63) / 64, p.wide[i]);
  if (p.splits[i] > 1) p.part[i] = at.take<float>(p.splits[i] * n * round_up(m, 4));
}

FfnPlan ffn_plan(int64_t rows, int64_t dim, int64_t hidden, int32_t dtype, bool backward,
                 void* ws) {
  FfnPlan p{};
  p.planes = dtype == SM_BF16 ? 1 : 3;
  p.ld_d = round_up(dim, 8);
  p.ld_f = round_up(hidden, 8);
  Places at{static_cast<char*>(ws)};
  if (!backward && rows <= kFewRows) {
    p.few_h = dtype == SM_BF16 ? (void*)at.take<bf16_t>(rows * hidden)
                               : (void*)at.take<float>(rows * hidden);
    p.bytes = at.used;
    return p;
  }
  const int64_t segs = p.planes == 1 ? 1 : 6;
  p.x = at.take<bf16_t>(p.planes * rows * p.ld_d);
  p.wg = at.take<bf16_t>(p.planes * hidden * p.ld_d);
  p.wu = at.take<bf16_t>(p.planes * hidden * p.ld_d);
  p.wd = at.take<bf16_t>(p.planes * dim * p.ld_f);
  p.h = at.take<bf16_t>(p.planes * rows * p.ld_f);
  if (!backward) {
    plan_product(p, at, 0, dim, rows, segs * hidden);
  } else {
    p.dy = at.take<bf16_t>(p.planes * rows * p.ld_d);
    p.dg = at.take<bf16_t>(p.planes * rows * p.ld_f);
    p.du = at.take<bf16_t>(p.planes * rows * p.ld_f);
    plan_product(p, at, 0, dim, rows, 2 * segs * hidden);
    plan_product(p, at, 1, dim, hidden, segs * rows);
    plan_product(p, at, 2, dim, hidden, segs * rows);
    plan_product(p, at, 3, hidden, dim, segs * rows);
  }
  p.bytes = at.used;
  return p;
}

hipError_t operand(Operand& o, const void* src, int32_t dtype, int64_t rows, int64_t cols,
                   int64_t stride, int planes, bf16_t* copy, hipStream_t s) {
  if (operand_fits(src, dtype, cols, stride)) {
    o = {static_cast<const char*>(src), stride, 0, nullptr};
    return hipSuccess;
  }
  const int64_t ld = round_up(cols, 8);
  o = {reinterpret_cast<const char*>(copy), ld, rows * ld * 2, copy};
  return launch_planes({src, stride, dtype, planes, rows, (int)cols, (int32_t)ld, nullptr, nullptr,
                        copy}, s);
}

MmJob product(const Operand& a, const Operand& b, int64_t m, int64_t n, int64_t k, int planes,
              int splits) {
  MmJob j{};
  j.a = a.p;
  j.b = b.p;
  j.lda = a.ld;
  j.ldb = b.ld;
  j.m = (int)m;
  j.n = (int)n;
  j.k = (int)k;
  j.splits = splits;
  set_planes(j, planes, a.plane, b.plane);
  return j;
}

// Where product i's results go: its sums of splits, or the caller's array.
MmOut out_of(const FfnPlan& p, int i, void* dst, int64_t m, int64_t n, int32_t dtype, int32_t add) {
  const int64_t ld = round_up(m, 4);
  if (p.splits[i] > 1) return {p.part[i], ld, n * ld, SM_F32, 0};
  return {dst, m, 0, dtype, add};
}
hipError_t join(const FfnPlan& p, int i, void* dst, int64_t m, int64_t n, int32_t dtype,
                int32_t add, hipStream_t s) {
  if (p.splits[i] <= 1) return hipSuccess;
  const int64_t ld = round_up(m, 4);
  return launch_join({p.part[i], n * ld, ld, p.splits[i], nullptr, n, (int)m, dtype, add, dst, m},
                     s);
}

template <typename T, int ACT>
hipError_t ffn_few(const FfnArgs& a, const FfnPlan& p, hipStream_t s) {
  const auto grid = [](int64_t m) {
    return dim3((unsigned)std::min<int64_t>((m + 15) / 16, 2 * kCus));
  };
  typedef FewGate<T, ACT> Gate;
  hipLaunchKernelGGL((k_few<T, 2, 8, Gate>), grid(a.hidden), dim3(512), 0, s, (const T*)a.Wg,
                     (const T*)a.Wu, a.dim, (int)a.hidden, (const T*)a.X, a.x_stride, (int)a.rows,
                     (const int32_t*)nullptr, (int)a.dim,
                     (typename Gate::Args{(T*)p.few_h, a.pre}));
  SM_TRY(hipGetLastError());
  hipLaunchKernelGGL((k_few<T, 1, 8, FewStore<T>>), grid(a.dim), dim3(512), 0, s, (const T*)a.Wd,
                     (const T*)nullptr, a.hidden, (int)a.dim, (const T*)p.few_h, a.hidden,
                     (int)a.rows, (const int32_t*)nullptr, (int)a.hidden,
                     (typename FewStore<T>::Args{(T*)a.Y}));
  return hipGetLastError();
}

template <int P, int ACT>
hipError_t ffn(const FfnArgs& a, hipStream_t s) {
  const FfnPlan p = ffn_plan(a.rows, a.dim, a.hidden, a.dtype, false, a.ws);
  if (a.rows <= kFewRows)
    return ffn_few<std::conditional_t<P == 1, bf16_t, float>, ACT>(a, p, s);
  Operand x, wg, wu, wd;
  SM_TRY(operand(x, a.X, a.dtype, a.rows, a.dim, a.x_stride, P, p.x, s));
  // both weights lie where they are, or both are copied: they share a row length
  const bool fits = operand_fits(a.Wg, a.dtype, a.dim, a.dim) &&
                    operand_fits(a.Wu, a.dtype, a.dim, a.dim);
  if (fits) {
    wg = {(const char*)a.Wg, a.dim, 0, nullptr};
    wu = {(const char*)a.Wu, a.dim, 0, nullptr};
  } else {
    const int64_t plane = a.hidden * p.ld_d * 2;
    wg = {(const char*)p.wg, p.ld_d, plane, p.wg};
    wu = {(const char*)p.wu, p.ld_d, plane, p.wu};
    for (auto [src, dst] : {std::pair{a.Wg, p.wg}, std::pair{a.Wu, p.wu}})
      SM_TRY(launch_planes({src, a.dim, a.dtype, P, a.hidden, (int)a.dim, (int32_t)p.ld_d, nullptr,
                            nullptr, dst}, s));
  }
  SM_TRY(operand(wd, a.Wd, a.dtype, a.dim, a.hidden, a.hidden, P, p.wd, s));
  MmArgs m{};
  m.jobs = 1;
  m.job[0] = product(wg, x, a.hidden, a.rows, a.dim, P, 1);
  m.job[0].a2 = wu.p;
  const int64_t plane = a.rows * p.ld_f;
  SM_TRY((run_mm<false, false, true, EpiGate<P, ACT>>(m, {p.h, p.ld_f, plane, a.pre},
                                                      wide_tiles(2 * a.hidden, a.rows), s)));
  const Operand h{(const char*)p.h, p.ld_f, plane * 2, nullptr};
  m = MmArgs{};
  m.jobs = 1;
  m.job[0] = product(wd, h, a.dim, a.rows, a.hidden, P, p.splits[0]);
  EpiStore::Args e{};
  e.out[0] = out_of(p, 0, a.Y, a.dim, a.rows, a.dtype, 0);
  SM_TRY((run_mm<false, false, false, EpiStore>(m, e, p.wide[0], s)));
  return join(p, 0, a.Y, a.dim, a.rows, a.dtype, 0, s);
}

template <int P, int ACT>
hipError_t ffn_grad(const FfnGradArgs& a, hipStream_t s) {
  const FfnPlan p = ffn_plan(a.rows, a.dim, a.hidden, a.dtype, true, a.ws);
  Operand x, dy, wg, wu, wd;
  SM_TRY(operand(dy, a.dY, a.dtype, a.rows, a.dim, a.dy_stride, P, p.dy, s));
  SM_TRY(operand(wd, a.Wd, a.dtype, a.dim, a.hidden, a.hidden, P, p.wd, s));
  const int64_t plane = a.rows * p.ld_f;
  MmArgs m{};
  m.jobs = 1;
  m.job[0] = product(wd, dy, a.hidden, a.rows, a.dim, P, 1);
  SM_TRY((run_mm<true, false, false, EpiGateGrad<P, ACT>>(
      m, {p.dg, p.du, p.h, p.ld_f, plane, a.pre}, wide_tiles(a.hidden, a.rows), s)));
  const Operand dg{(const char*)p.dg, p.ld_f, plane * 2, nullptr};
  const Operand du{(const char*)p.du, p.ld_f, plane * 2, nullptr};
  const Operand h{(const char*)p.h, p.ld_f, plane * 2, nullptr};
  if (a.dX) {
    SM_TRY(operand(wg, a.Wg, a.dtype, a.hidden, a.dim, a.dim, P, p.wg, s));
    SM_TRY(operand(wu, a.Wu, a.dtype, a.hidden, a.dim, a.dim, P, p.wu, s));
    if (wg.copy == nullptr && wu.copy != nullptr) {      // one row length for both
      wg = {(const char*)p.wg, p.ld_d, wu.plane, p.wg};
      SM_TRY(launch_planes({a.Wg, a.dim, a.dtype, P, a.hidden, (int)a.dim, (int32_t)p.ld_d,
                            nullptr, nullptr, p.wg}, s));
    }
    m = MmArgs{};
    m.jobs = 1;
    m.job[0] = product(wg, dg, a.dim, a.rows, a.hidden, P, p.splits[0]);
    m.job[0].parts = 2;
    m.job[0].a_part = wu.p - wg.p;
    m.job[0].b_part = du.p - dg.p;
    EpiStore::Args e{};
    e.out[0] = out_of(p, 0, a.dX, a.dim, a.rows, a.dtype, 0);
    SM_TRY((run_mm<true, false, false, EpiStore>(m, e, p.wide[0], s)));
    SM_TRY(join(p, 0, a.dX, a.dim, a.rows, a.dtype, 0, s));
  }
  if (!a.dWg && !a.dWu && !a.dWd) return hipSuccess;
  if (a.dWg || a.dWu) SM_TRY(operand(x, a.X, a.dtype, a.rows, a.dim, a.x_stride, P, p.x, s));
  m = MmArgs{};
  EpiStore::Args e{};
  const auto add = [&](int i, const Operand& A, const Operand& B, void* dst, int64_t mm,
                       int64_t nn) {
    if (!dst) return;
    e.out[m.jobs] = out_of(p, i, dst, mm, nn, a.dw_dtype, a.accumulate);
    m.job[m.jobs++] = product(A, B, mm, nn, a.rows, P, p.splits[i]);
  };
  add(1, x, dg, a.dWg, a.dim, a.hidden);
  add(2, x, du, a.dWu, a.dim, a.hidden);
  add(3, h, dy, a.dWd, a.hidden, a.dim);
  SM_TRY((run_mm<true, true, false, EpiStore>(m, e, p.wide[1], s)));
  if (a.dWg) SM_TRY(join(p, 1, a.dWg, a.dim, a.hidden, a.dw_dtype, a.accumulate, s));
  if (a.dWu) SM_TRY(join(p, 2, a.dWu, a.dim, a.hidden, a.dw_dtype, a.accumulate, s));
  if (a.dWd) SM_TRY(join(p, 3, a.dWd, a.hidden, a.dim, a.dw_dtype, a.accumulate, s));
  return hipSuccess;
}

}  // namespace

size_t ffn_workspace(int64_t rows, int64_t dim, int64_t hidden, int32_t dtype, bool backward) {
  return rows == 0 ? 0 : ffn_plan(rows, dim, hidden, dtype, backward, nullptr).bytes;
}

hipError_t launch_ffn(const FfnArgs& a, hipStream_t s) {
  if (a.dtype == SM_BF16) return a.act == 0 ? ffn<1, 0>(a, s) : ffn<1, 1>(a, s);
  return a.act == 0 ? ffn<3, 0>(a, s) : ffn<3, 1>(a, s);
}

hipError_t launch_ffn_grad(const FfnGradArgs& a, hipStream_t s) {
  if (a.rows == 0) {           // sums of nothing
    if (a.accumulate) return hipSuccess;
    for (void* p : {a.dWg, a.dWu, a.dWd})
      if (p) SM_TRY(launch_zero(p, a.dw_dtype, a.dim * a.hidden, s));
    return hipSuccess;
  }
  if (a.dtype == SM_BF16) return a.act == 0 ? ffn_grad<1, 0>(a, s) : ffn_grad<1, 1>(a, s);
  return a.act == 0 ? ffn_grad<3, 0>(a, s) : ffn_grad<3, 1>(a, s);
}

}  // namespace sm
