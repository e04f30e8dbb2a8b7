// Embedding lookup and the gradient of its table (signmuon_layers.h).  The
// gradient sorts the tokens (stably, so that the rows of one token are added
// in their order in the batch) and sums the rows of each token; integer
// counts only, no floating-point atomics.  All of it is bound by HBM: the rows
// that are read, and above all the table's gradient that is written.
#include <algorithm>

#include "sm_layers.h"
#include "sm_rows.h"

namespace sm {

// ---------------------------------------------------------------------------
// Lookup: LANES threads a row, which moves in pieces of V entries (16 bytes of
// the narrower type).  The piece that would pass the row's end starts earlier
// instead and copies some entries twice; rows shorter than a piece go entry
// by entry (V = 1).
// ---------------------------------------------------------------------------
template <typename TW, typename TY, typename TI, int V, int LANES>
__global__ __launch_bounds__(256) void k_embed(const TW* __restrict__ W, int64_t vocab, int dim,
                                               const TI* __restrict__ tokens, int64_t n,
                                               float scale, TY* __restrict__ Y) {
  constexpr int GROUPS = 256 / LANES;
  const int lane = threadIdx.x % LANES;
  for (int64_t i = (int64_t)blockIdx.x * GROUPS + threadIdx.x / LANES; i < n;
       i += (int64_t)gridDim.x * GROUPS) {
    const int64_t t = tokens[i];
    const bool ok = t >= 0 && t < vocab;
    const TW* w = W + (ok ? t : 0) * dim;
    TY* y = Y + i * dim;
#pragma unroll 2
    for (int c0 = lane * V; c0 < dim; c0 += LANES * V) {
      const int c = c0 + V <= dim ? c0 : dim - V;
      float v[V];
      if constexpr (V == 1) v[0] = to_f32(w[c]);
      else load_vec<V>(w + c, v);
#pragma unroll
      for (int k = 0; k < V; ++k) v[k] = ok ? scale * v[k] : __builtin_nanf("");
      if constexpr (V == 1) put(y + c, v[0]);
      else store_vec<V>(y + c, v);
    }
  }
}

// ---------------------------------------------------------------------------
// Sort.  Block b owns the tokens lo <= t < lo + range and reads the whole
// batch, so the blocks need nothing of each other: tokens below lo are counted
// on the way, which gives the block's place in the sorted order.  Each of its
// 16 waves reads one run of consecutive positions and lists the positions it
// finds in range, in order; the list is counted by token, the counts are
// scanned over tokens and waves, and the list is placed.  A wave whose list
// overflows counts it and starts it anew, and reads its run again to place.
// Equal tokens among 64 listed ones are found by one ballot per bit of t - lo.
// Between counting and placing the block clears the rows of the table that no
// token names (unless the caller accumulates), while placing goes on.
//   order[p], sorted[p]: batch position and token of the p-th in sorted order
//   start[v]: the first p of token v; start[vocab]: how many tokens count
// One launch.  Every block reading all tokens costs n / 64 loads a wave run
// (n = 65536: 8 us) and grows with n; a sort by digits would read each token
// once a pass but takes two launches a pass.
// ---------------------------------------------------------------------------
constexpr int kSortWaves = 16;
constexpr int kMaxRange = 512;   // 32 KB of counts
constexpr int kList = 256;       // listed positions a wave

template <typename TI, typename TO>
__global__ __launch_bounds__(64 * kSortWaves) void k_token_sort(
    const TI* __restrict__ tokens, int64_t n, int64_t vocab, int64_t padding, int range, int bits,
    int32_t* __restrict__ order, int32_t* __restrict__ sorted, int32_t* __restrict__ start,
    TO* __restrict__ dW, int dim) {
  extern __shared__ int32_t counts[];   // [kSortWaves][range]
  __shared__ int32_t list_pos[kSortWaves][kList];
  __shared__ uint16_t list_bin[kSortWaves][kList];
  __shared__ int32_t below[kSortWaves], wave_total[kSortWaves];
  __shared__ uint8_t empty[kMaxRange];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint64_t before = ((uint64_t)1 << lane) - 1;
  const int64_t lo = (int64_t)blockIdx.x * range;
  const int64_t share = ((n + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;
  const int64_t i0 = w * share, i1 = i0 + share < n ? i0 + share : n;
  volatile int32_t* mine = counts + w * range;
  volatile int32_t* pos = list_pos[w];
  volatile uint16_t* bin = list_bin[w];
  for (int k = threadIdx.x; k < kSortWaves * range; k += 64 * kSortWaves) counts[k] = 0;
  __syncthreads();

  // Counts (or, once the counts hold places, places) the first `len` listed.
  auto settle = [&](int len, bool place) {
    for (int k = 0; k < len; k += 64) {
      const bool in = k + lane < len;
      const int b = in ? bin[k + lane] : 0;
      uint64_t peers = __ballot(in);
      for (int d = 0; d < bits; ++d) {
        const bool set = (b >> d) & 1;
        const uint64_t v = __ballot(set);
        peers &= set ? v : ~v;
      }
      if (in) {
        const int32_t c = mine[b];
        if (place) {
          const int32_t p = c + __popcll(peers & before);
          order[p] = pos[k + lane];
          sorted[p] = (int32_t)(lo + b);
        }
        __builtin_amdgcn_wave_barrier();
        if ((peers & before) == 0) mine[b] = c + __popcll(peers);
      }
      __builtin_amdgcn_wave_barrier();
    }
  };
  // Lists the wave's run, settling full lists; returns what is still listed.
  bool whole = true;      // the list holds all of the wave's positions
  int32_t under = 0;
  auto scan = [&](bool place) {
    int len = 0;
    constexpr int U = 8;      // loads in flight
    for (int64_t i = i0; i < i1; i += 64 * U) {
      int64_t t[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t at = i + 64 * u + lane;
        t[u] = at < i1 ? (int64_t)tokens[at] : -1;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool valid = t[u] >= 0 && t[u] < vocab && t[u] != padding;
        const bool in = valid && t[u] >= lo && t[u] < lo + range;
        under += __popcll(__ballot(valid && t[u] < lo));
        const uint64_t m = __ballot(in);
        if (m == 0) continue;
        const int more = __popcll(m);
        if (len + more > kList) {
          settle(len, place);
          whole = false;
          len = 0;
        }
        if (in) {
          const int at = len + __popcll(m & before);
          pos[at] = (int32_t)(i + 64 * u + lane);
          bin[at] = (uint16_t)(t[u] - lo);
        }
        len += more;
      }
    }
    return len;
  };

  int len = scan(false);
  settle(len, false);
  if (lane == 0) below[w] = under;
  __syncthreads();
  // thread k holds token lo + k (range <= the threads of the block)
  const int mybin = threadIdx.x;
  int32_t base = 0;
  for (int k = 0; k < kSortWaves; ++k) base += below[k];
  int32_t total = 0;
  if (mybin < range)
    for (int k = 0; k < kSortWaves; ++k) total += counts[k * range + mybin];
  int32_t incl = total;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int32_t up = __shfl_up(incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 63) wave_total[w] = incl;
  __syncthreads();
  for (int k = 0; k < w; ++k) base += wave_total[k];
  if (mybin < range) {
    int32_t at = base + incl - total;
    if (lo + mybin < vocab) start[lo + mybin] = at;
    if (lo + mybin == vocab - 1) start[vocab] = at + total;
    empty[mybin] = total == 0 && lo + mybin < vocab;
    for (int k = 0; k < kSortWaves; ++k) {
      const int32_t c = counts[k * range + mybin];
      counts[k * range + mybin] = at;
      at += c;
    }
  }
  __syncthreads();
  if (dW) {
    constexpr int V = 16 / (int)sizeof(TO);
    const float zero[V] = {};
    const int pieces = (dim + V - 1) / V;
    int lanes = 64;                       // threads a row
    while (lanes > 1 && lanes >= 2 * pieces) lanes >>= 1;
    const int rows = 64 / lanes;
    for (int r = w * rows + lane / lanes; r < range; r += kSortWaves * rows)
      if (empty[r]) {
        TO* row = dW + (lo + r) * dim;
        for (int c = lane % lanes * V; c < dim; c += lanes * V) store_part<V>(row + c, dim - c, zero);
      }
  }
  if (!whole) len = scan(true);
  settle(len, true);
}

// ---------------------------------------------------------------------------
// Sums.  The sorted positions are cut into units of `span` positions, one wave
// each (and each slice of 64 V columns).  A unit finishes the tokens that
// begin in it, even past its end, unless a token has more than kLong rows:
// of those every unit sums its own positions only, to part[2 u] where the
// token began before the unit and part[2 u + 1] where it begins in it, and
// k_embed_join adds the parts.  So work is even however often a token occurs
// (a unit adds at most span + kLong rows) and most rows need no second pass.
// ---------------------------------------------------------------------------
constexpr int kLong = 64;    // at least the span

template <int V, typename T>
__device__ __forceinline__ void read_cols(const T* p, float (&v)[V]) {
  if constexpr (V == 1) v[0] = to_f32(*p);
  else load_vec<V>(p, v);
}

template <typename T, typename TO, int V>
__global__ __launch_bounds__(256) void k_embed_sum(
    const T* __restrict__ dY, int64_t dys, const int32_t* __restrict__ order,
    const int32_t* __restrict__ sorted, const int32_t* __restrict__ start, int64_t vocab, int dim,
    int slices, int span, float scale, TO* __restrict__ dW, int accumulate,
    float* __restrict__ part) {
  constexpr int U = 8;      // rows in flight
  const int lane = threadIdx.x & 63;
  const int64_t wave = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t unit = wave / slices;
  const int64_t p0 = unit * span, n = start[vocab];
  if (p0 >= n) return;
  const int64_t p1 = p0 + span < n ? p0 + span : n;
  // columns; a lane that would pass the row's end starts earlier and leaves
  // the `skip` entries before its own to the lane that has them
  int c = ((int)(wave - unit * slices) * 64 + lane) * V, skip = 0;
  if (c >= dim) skip = V;
  else if (c + V > dim) skip = c + V - dim;
  c = c + V <= dim ? c : dim - V;

  int64_t p = p0, end = p1;
  const int32_t first = sorted[p0], last = sorted[p1 - 1];
  const int32_t s1 = start[first], e1 = start[first + 1];
  const int32_t s2 = start[last], e2 = start[last + 1];
  bool head = false, tail = false;      // the first / last token's rows are a part
  if (s1 < p0) {
    if (e1 - s1 > kLong) head = true;
    else p = e1;
  }
  if (e2 > p1) {
    if (e2 - s2 > kLong) tail = true;
    else end = e2;
  }
  if (p >= end) return;
  float acc[V];
#pragma unroll
  for (int k = 0; k < V; ++k) acc[k] = 0.f;
  int32_t cur = __builtin_amdgcn_readfirstlane(sorted[p]);
  auto flush = [&](bool is_last) {
    if (skip < V) {
      if (head || (is_last && tail)) {
        float* out = part + (2 * unit + (head ? 0 : 1)) * dim + c;
#pragma unroll
        for (int k = 0; k < V; ++k)
          if (k >= skip) out[k] = acc[k];
      } else {
        TO* out = dW + (int64_t)cur * dim + c;
        float v[V];
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = scale * acc[k];
        if (accumulate) {
          float old[V];
          read_cols<V>(out, old);
#pragma unroll
          for (int k = 0; k < V; ++k) v[k] += old[k];
        }
        if constexpr (V > 1) {
          if (skip == 0) store_vec<V>(out, v);
        }
        if (V == 1 || skip > 0)
#pragma unroll
          for (int k = 0; k < V; ++k)
            if (k >= skip) put(out + k, v[k]);
      }
    }
    head = false;
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.f;
  };
  for (; p < end; p += 64) {
    const int have = (int)(end - p < 64 ? end - p : 64);
    const int32_t row = lane < have ? order[p + lane] : 0;
    const int32_t tok = lane < have ? sorted[p + lane] : 0;
    for (int i = 0; i < have; i += U) {
      float v[U][V];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t r = __builtin_amdgcn_readlane(row, i + u < have ? i + u : i);
        read_cols<V>(dY + r * dys + c, v[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + u < have) {
          const int32_t t = __builtin_amdgcn_readlane(tok, i + u);
          if (t != cur) {
            flush(false);
            cur = t;
          }
#pragma unroll
          for (int k = 0; k < V; ++k) acc[k] += v[u][k];
        }
    }
  }
  flush(true);
}

// Adds the parts of long tokens.  A block looks for the long tokens that begin
// in its kJoinUnits units; its 8 waves each add a run of consecutive parts
// (64 columns), and meet in LDS.
constexpr int kJoinUnits = 16, kJoinWaves = 8;

template <typename TO>
__global__ __launch_bounds__(64 * kJoinWaves) void k_embed_join(
    const float* __restrict__ part, const int32_t* __restrict__ sorted,
    const int32_t* __restrict__ start, int64_t vocab, int dim, int span, float scale,
    TO* __restrict__ dW, int accumulate) {
  __shared__ float sh[kJoinWaves][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int c = blockIdx.y * 64 + lane;
  const int64_t n = start[vocab];
  for (int k = 0; k < kJoinUnits; ++k) {
    const int64_t u = (int64_t)blockIdx.x * kJoinUnits + k, p0 = u * span;
    if (p0 + span >= n) return;           // nothing goes on past this unit
    const int32_t t = sorted[p0 + span - 1];
    const int32_t s = start[t], e = start[t + 1];
    if (s < p0 || e <= p0 + span || e - s <= kLong) continue;
    // part 2u + 1, then 2j for the units j after u up to the token's end
    const int64_t parts = (e - 1) / span - u + 1;
    const int64_t run = (parts + kJoinWaves - 1) / kJoinWaves;
    const int64_t j1 = (w + 1) * run < parts ? (w + 1) * run : parts;
    float a = 0.f;
    if (c < dim) {
#pragma unroll 8
      for (int64_t j = w * run; j < j1; ++j)
        a += part[(2 * (u + j) + (j == 0)) * dim + c];
    }
    sh[w][lane] = a;
    __syncthreads();
    if (w == 0 && c < dim) {
#pragma unroll
      for (int q = 1; q < kJoinWaves; ++q) a += sh[q][lane];
      TO* out = dW + (int64_t)t * dim + c;
      put(out, accumulate ? to_f32(*out) + scale * a : scale * a);
    }
    __syncthreads();
  }
}

namespace {

constexpr int64_t kMaxBlocks = 1 << 16;   // larger grids loop

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Positions a unit.
int span_of(int64_t n) { return n <= 32768 ? 16 : 32; }

struct GradPlan {
  int span, range, bits;
  int64_t units;
  size_t order, sorted, start, part, total;
  GradPlan(int64_t n, int64_t vocab, int64_t dim) {
    range = (int)std::min<int64_t>((vocab + 255) / 256, kMaxRange);
    for (bits = 0; (1 << bits) < range;) ++bits;
    span = span_of(n);
    units = (n + span - 1) / span;
    order = 0;
    sorted = order + align256((size_t)n * 4);
    start = sorted + align256((size_t)n * 4);
    part = start + align256((size_t)(vocab + 1) * 4);
    // no token has more than kLong rows in a batch of kLong
    total = part + (n > kLong ? align256((size_t)units * 2 * dim * 4) : 0);
  }
};

template <typename TW, typename TY, typename TI, int V, int LANES>
void embed_go(const EmbedArgs& a, hipStream_t s) {
  const int64_t groups = 256 / LANES;
  const int64_t grid = std::min<int64_t>((a.n + groups - 1) / groups, kMaxBlocks);
  hipLaunchKernelGGL((k_embed<TW, TY, TI, V, LANES>), dim3((unsigned)grid), dim3(256), 0, s,
                     (const TW*)a.W, a.vocab, (int)a.dim, (const TI*)a.tokens, a.n, a.scale,
                     (TY*)a.Y);
}

template <typename TW, typename TY, typename TI>
void embed_lanes(const EmbedArgs& a, hipStream_t s) {
  constexpr int V = sizeof(TW) == 4 && sizeof(TY) == 4 ? 4 : 8;
  if (a.dim < V) embed_go<TW, TY, TI, 1, 4>(a, s);
  else if (a.dim <= 8 * V) embed_go<TW, TY, TI, V, 8>(a, s);
  else embed_go<TW, TY, TI, V, 64>(a, s);
}

template <typename TW, typename TY>
hipError_t embed(const EmbedArgs& a, hipStream_t s) {
  if (a.token_bits == 64) embed_lanes<TW, TY, int64_t>(a, s);
  else embed_lanes<TW, TY, int32_t>(a, s);
  return hipGetLastError();
}

template <typename TI, typename TO>
hipError_t token_sort(const EmbedGradArgs& a, const GradPlan& pl, int32_t* order, int32_t* sorted,
                      int32_t* start, hipStream_t s) {
  const int64_t grid = (a.vocab + pl.range - 1) / pl.range;
  hipLaunchKernelGGL((k_token_sort<TI, TO>), dim3((unsigned)grid), dim3(64 * kSortWaves),
                     (size_t)kSortWaves * pl.range * 4, s, (const TI*)a.tokens, a.n, a.vocab,
                     a.padding, pl.range, pl.bits, order, sorted, start,
                     a.accumulate ? nullptr : (TO*)a.dW, (int)a.dim);
  return hipGetLastError();
}

template <typename T, typename TO, int V>
void embed_sum(const EmbedGradArgs& a, const GradPlan& pl, const int32_t* order,
               const int32_t* sorted, const int32_t* start, float* part, hipStream_t s) {
  const int64_t slices = (a.dim + 64 * V - 1) / (64 * V);
  hipLaunchKernelGGL((k_embed_sum<T, TO, V>), dim3((unsigned)((pl.units * slices + 3) / 4)),
                     dim3(256), 0, s, (const T*)a.dY, a.dy_stride, order, sorted, start, a.vocab,
                     (int)a.dim, (int)slices, pl.span, a.scale, (TO*)a.dW, a.accumulate, part);
}

template <typename T, typename TO>
hipError_t embed_grad(const EmbedGradArgs& a, hipStream_t s) {
  const GradPlan pl(a.n, a.vocab, a.dim);
  char* ws = (char*)a.ws;
  int32_t* order = (int32_t*)(ws + pl.order);
  int32_t* sorted = (int32_t*)(ws + pl.sorted);
  int32_t* start = (int32_t*)(ws + pl.start);
  float* part = (float*)(ws + pl.part);
  hipError_t e = a.token_bits == 64 ? token_sort<int64_t, TO>(a, pl, order, sorted, start, s)
                                    : token_sort<int32_t, TO>(a, pl, order, sorted, start, s);
  if (e != hipSuccess || a.n == 0) return e;
  if (sizeof(T) == 2 && a.dim >= 512)
    embed_sum<T, TO, 8>(a, pl, order, sorted, start, part, s);
  else if (a.dim >= 4)
    embed_sum<T, TO, 4>(a, pl, order, sorted, start, part, s);
  else
    embed_sum<T, TO, 1>(a, pl, order, sorted, start, part, s);
  if ((e = hipGetLastError()) != hipSuccess || a.n <= kLong) return e;
  hipLaunchKernelGGL((k_embed_join<TO>),
                     dim3((unsigned)((pl.units + kJoinUnits - 1) / kJoinUnits),
                          (unsigned)((a.dim + 63) / 64)),
                     dim3(64 * kJoinWaves), 0, s, part, sorted, start, a.vocab, (int)a.dim,
                     pl.span, a.scale, (TO*)a.dW, a.accumulate);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_embed(const EmbedArgs& a, hipStream_t s) {
  if (a.w_dtype == SM_BF16)
    return a.y_dtype == SM_BF16 ? embed<bf16_t, bf16_t>(a, s) : embed<bf16_t, float>(a, s);
  return a.y_dtype == SM_BF16 ? embed<float, bf16_t>(a, s) : embed<float, float>(a, s);
}

size_t embed_grad_workspace(int64_t n, int64_t vocab, int64_t dim) {
  return GradPlan(n, vocab, dim).total;
}

hipError_t launch_embed_grad(const EmbedGradArgs& a, hipStream_t s) {
  if (a.dy_dtype == SM_BF16)
    return a.dw_dtype == SM_BF16 ? embed_grad<bf16_t, bf16_t>(a, s)
                                 : embed_grad<bf16_t, float>(a, s);
  return a.dw_dtype == SM_BF16 ? embed_grad<float, bf16_t>(a, s) : embed_grad<float, float>(a, s);
}

}  // namespace sm
