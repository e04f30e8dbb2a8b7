// Embedding lookup and the gradient of its table (signmuon_layers.h).  The
// gradient sorts the tokens (stably, so that the rows of one token are added
// in their order in the batch) and sums the rows of each token; integer
// counts only, no floating-point atomics.
#include "sm_layers.h"
#include "sm_rows.h"

namespace sm {

// ---------------------------------------------------------------------------
// Lookup: one block per row.
// ---------------------------------------------------------------------------
template <typename TW, typename TY, typename TI>
__global__ __launch_bounds__(256) void k_embed(const TW* W, int64_t vocab, int dim,
                                               const TI* tokens, int64_t n, float scale, TY* Y) {
  for (int64_t i = blockIdx.x; i < n; i += gridDim.x) {
    const int64_t t = tokens[i];
    const bool ok = t >= 0 && t < vocab;
    const TW* w = W + (ok ? t : 0) * dim;
    TY* y = Y + i * dim;
    for (int c = threadIdx.x; c < dim; c += 256)
      put(y + c, ok ? scale * to_f32(w[c]) : __builtin_nanf(""));
  }
}

// ---------------------------------------------------------------------------
// Sort.  Block b owns the tokens lo = b * range <= t < lo + range and reads
// the whole batch: its 16 waves each take one run of consecutive positions,
// first to count their tokens of every value, then, from the scanned counts,
// to place the positions.  Tokens below lo are counted on the way: they are
// the block's own offset, so the blocks need nothing of each other.  Equal
// tokens of 64 positions are found by one ballot per bit of t - lo.
//   perm[p]: the batch position of the p-th token in sorted order
//   start[v]: the first p of token v; start[vocab]: how many tokens count
// ---------------------------------------------------------------------------
constexpr int kSortWaves = 16;
constexpr int kMaxRange = 512;   // 32 KB of counts

struct Match {
  uint64_t in;      // lanes whose token lies in the block's range
  uint64_t below;   // lanes whose token counts and lies below it
  uint64_t peers;   // lanes of `in` with this lane's token
  int bin;          // token - lo, where in range
};

template <typename TI>
__device__ __forceinline__ Match match(const TI* tokens, int64_t i, int64_t n, int64_t vocab,
                                       int64_t padding, int64_t lo, int range, int bits) {
  const int64_t t = i < n ? (int64_t)tokens[i] : -1;
  const bool valid = t >= 0 && t < vocab && t != padding;
  Match m;
  m.in = __ballot(valid && t >= lo && t < lo + range);
  m.below = __ballot(valid && t < lo);
  m.bin = (int)(t - lo);
  m.peers = m.in;
  if (m.in)
    for (int b = 0; b < bits; ++b) {
      const bool set = (m.bin >> b) & 1;
      const uint64_t v = __ballot(set);
      m.peers &= set ? v : ~v;
    }
  return m;
}

template <typename TI>
__global__ __launch_bounds__(64 * kSortWaves) void k_token_sort(
    const TI* tokens, int64_t n, int64_t vocab, int64_t padding, int range, int bits,
    int32_t* perm, int32_t* start) {
  extern __shared__ int32_t counts[];   // [kSortWaves][range]
  __shared__ int32_t below[kSortWaves], wave_total[kSortWaves];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t lo = (int64_t)blockIdx.x * range;
  const int64_t share = ((n + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;
  const int64_t i0 = w * share, i1 = i0 + share < n ? i0 + share : n;
  volatile int32_t* mine = counts + w * range;
  for (int k = threadIdx.x; k < kSortWaves * range; k += 64 * kSortWaves) counts[k] = 0;
  __syncthreads();
  int32_t under = 0;
  for (int64_t i = i0; i < i1; i += 64) {
    const Match m = match(tokens, i + lane, n, vocab, padding, lo, range, bits);
    under += __popcll(m.below);
    if ((m.in >> lane & 1) && lane == __ffsll((unsigned long long)m.peers) - 1)
      mine[m.bin] = mine[m.bin] + __popcll(m.peers);
  }
  if (lane == 0) below[w] = under;
  __syncthreads();
  // thread k holds bin k (range <= the threads of the block)
  int32_t base = 0;
  for (int k = 0; k < kSortWaves; ++k) base += below[k];
  int32_t total = 0;
  if ((int)threadIdx.x < range)
    for (int k = 0; k < kSortWaves; ++k) total += counts[k * range + threadIdx.x];
  int32_t incl = total;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int32_t up = __shfl_up(incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 63) wave_total[w] = incl;
  __syncthreads();
  for (int k = 0; k < w; ++k) base += wave_total[k];
  int32_t at = base + incl - total;
  if ((int)threadIdx.x < range) {
    if (lo + threadIdx.x < vocab) start[lo + threadIdx.x] = at;
    if (lo + threadIdx.x == vocab - 1) start[vocab] = at + total;
    for (int k = 0; k < kSortWaves; ++k) {
      const int32_t c = counts[k * range + threadIdx.x];
      counts[k * range + threadIdx.x] = at;
      at += c;
    }
  }
  __syncthreads();
  for (int64_t i = i0; i < i1; i += 64) {
    const Match m = match(tokens, i + lane, n, vocab, padding, lo, range, bits);
    if (m.in >> lane & 1) {
      const int32_t p = mine[m.bin];
      perm[p + __popcll(m.peers & ((1ull << lane) - 1))] = (int32_t)(i + lane);
      __builtin_amdgcn_wave_barrier();
      if (lane == __ffsll((unsigned long long)m.peers) - 1)
        mine[m.bin] = p + __popcll(m.peers);
    }
  }
}

// One block per row of the table: its tokens' rows in sorted order.
template <typename T, typename TO>
__global__ __launch_bounds__(256) void k_embed_rows(const T* dY, int64_t dys,
                                                    const int32_t* perm, const int32_t* start,
                                                    int64_t vocab, int dim, float scale, TO* dW,
                                                    int accumulate) {
  for (int64_t v = blockIdx.x; v < vocab; v += gridDim.x) {
    const int32_t p0 = start[v], p1 = start[v + 1];
    if (accumulate && p0 == p1) continue;
    TO* out = dW + v * dim;
    for (int c = threadIdx.x; c < dim; c += 256) {
      float s = 0.f;
      for (int32_t p = p0; p < p1; ++p) s += to_f32(dY[perm[p] * dys + c]);
      put(out + c, accumulate ? to_f32(out[c]) + scale * s : scale * s);
    }
  }
}

namespace {

constexpr int64_t kMaxBlocks = 1 << 16;   // larger grids loop

int sort_range(int64_t vocab) {
  int64_t r = (vocab + 255) / 256;
  return (int)(r < kMaxRange ? r : kMaxRange);
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

struct GradPlan {
  size_t perm, start, total;
  GradPlan(int64_t n, int64_t vocab, int64_t) {
    perm = 0;
    start = align256((size_t)n * 4);
    total = start + align256((size_t)(vocab + 1) * 4);
  }
};

template <typename TW, typename TY>
hipError_t embed(const EmbedArgs& a, hipStream_t s) {
  const int64_t grid = a.n < kMaxBlocks ? a.n : kMaxBlocks;
  if (a.token_bits == 64)
    hipLaunchKernelGGL((k_embed<TW, TY, int64_t>), dim3((unsigned)grid), dim3(256), 0, s,
                       (const TW*)a.W, a.vocab, (int)a.dim, (const int64_t*)a.tokens, a.n,
                       a.scale, (TY*)a.Y);
  else
    hipLaunchKernelGGL((k_embed<TW, TY, int32_t>), dim3((unsigned)grid), dim3(256), 0, s,
                       (const TW*)a.W, a.vocab, (int)a.dim, (const int32_t*)a.tokens, a.n,
                       a.scale, (TY*)a.Y);
  return hipGetLastError();
}

template <typename TI>
hipError_t token_sort(const EmbedGradArgs& a, int32_t* perm, int32_t* start, hipStream_t s) {
  const int range = sort_range(a.vocab);
  int bits = 0;
  while ((1 << bits) < range) ++bits;
  const int64_t grid = (a.vocab + range - 1) / range;
  hipLaunchKernelGGL((k_token_sort<TI>), dim3((unsigned)grid), dim3(64 * kSortWaves),
                     (size_t)kSortWaves * range * 4, s, (const TI*)a.tokens, a.n, a.vocab,
                     a.padding, range, bits, perm, start);
  return hipGetLastError();
}

template <typename T, typename TO>
hipError_t embed_rows(const EmbedGradArgs& a, const int32_t* perm, const int32_t* start,
                      hipStream_t s) {
  const int64_t grid = a.vocab < kMaxBlocks ? a.vocab : kMaxBlocks;
  hipLaunchKernelGGL((k_embed_rows<T, TO>), dim3((unsigned)grid), dim3(256), 0, s,
                     (const T*)a.dY, a.dy_stride, perm, start, a.vocab, (int)a.dim, a.scale,
                     (TO*)a.dW, a.accumulate);
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
  const GradPlan pl(a.n, a.vocab, a.dim);
  int32_t* perm = (int32_t*)((char*)a.ws + pl.perm);
  int32_t* start = (int32_t*)((char*)a.ws + pl.start);
  hipError_t e = a.token_bits == 64 ? token_sort<int64_t>(a, perm, start, s)
                                    : token_sort<int32_t>(a, perm, start, s);
  if (e != hipSuccess) return e;
  if (a.dy_dtype == SM_BF16)
    return a.dw_dtype == SM_BF16 ? embed_rows<bf16_t, bf16_t>(a, perm, start, s)
                                 : embed_rows<bf16_t, float>(a, perm, start, s);
  return a.dw_dtype == SM_BF16 ? embed_rows<float, bf16_t>(a, perm, start, s)
                               : embed_rows<float, float>(a, perm, start, s);
}

}  // namespace sm
