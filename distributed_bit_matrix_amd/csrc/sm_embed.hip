// Embedding lookup and the gradient of its table (signmuon_layers.h).  The
// gradient sorts the tokens (stably, so that the rows of one token are added
// in their order in the batch) and sums the rows of each token; integer
// counts only, no floating-point atomics.  All of it is bound by HBM: the rows
// that are read, and above all the table's gradient that is written.
#include <algorithm>
#include <type_traits>

#include "sm_layers.h"
#include "sm_rows.h"

namespace sm {

// ---------------------------------------------------------------------------
// Lookup: LANES threads a row, which moves in pieces of V entries (16 bytes of
// the narrower type).  The piece that would pass the row's end starts earlier
// instead and copies some entries twice; rows shorter than a piece go entry
// by entry (V = 1).  12288 rows of 768 bfloat16 take 8.1 us.
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
      Piece<TW, V> p;
      p.load(w + c);
      float v[V];
#pragma unroll
      for (int k = 0; k < V; ++k) v[k] = ok ? scale * p[k] : __builtin_nanf("");
      store_vec<V>(y + c, v);
    }
  }
}

// ---------------------------------------------------------------------------
// Sort.  Equal tokens have to be neighbours, in the order of the batch; the
// tokens themselves may come in any fixed order.  Of B = 2^shift sets of
// blocks, set b takes the tokens t with t % B = b, so that frequent tokens,
// which vocabularies number next to each other, spread over the sets.
//
// Small batches (kOneLaunch): one block a set and one launch.  Every block
// reads the whole batch and needs nothing of the others: it counts the tokens
// of the sets before it on the way, which gives its place in the order.
// Larger ones (kRuns, kLongRuns): a set has a block for each of S runs of the
// batch; a first launch (k_token_count) counts every block's tokens, the
// second one knows from these counts where each token of each run goes.
//
// Each of a block's 16 waves reads a part of its run and lists the positions
// that are the set's; the list is counted by token, the counts are scanned
// over tokens and waves, and the list is placed.  A wave whose list overflows
// counts it and starts it anew, and reads its part again to place.  When
// placing, equal tokens among 64 listed ones are found by one ballot per bit
// of t / B.  Between counting and placing the block clears the rows of the
// table that no token names (unless the caller accumulates): those stores
// drain while placing goes on.
//   order[p], sorted[p]: batch position and token of the p-th in sorted order
//   total: how many tokens count
// Bound by the clearing where the table is large (131072 x 2048 float32: 912 MB
// in 160 to 180 us; 50257 x 768: 140 MB in 25 us), else by the instructions
// that look at every token in every block, 5 to 7 for 64 of them: 65536 tokens
// take 15 us in 256 blocks, 15.5 in 128 and 18 in 64.
// ---------------------------------------------------------------------------
constexpr int kSortWaves = 16;
constexpr int kBatch = 8;        // loads of 64 tokens in flight a wave
constexpr int kList = 64 * kBatch;   // listed positions a wave
constexpr int kRunBits = 16;     // a listed position: bin << 16 | place in the part
constexpr int kOneRange = 512, kOneShift = 8;   // one launch: tokens a block, fewest sets
constexpr int kSplitRange = 2048;               // two launches
constexpr int kWideRange = 1024;                // two launches over long runs

typedef volatile __attribute__((address_space(3))) uint32_t lds_u32;
typedef volatile __attribute__((address_space(3))) uint16_t lds_u16;

// A token as loaded: its low word, and whether that is all of it (a negative
// or larger token is no token of the table).
struct Token32 {
  uint32_t lo;
  __device__ __forceinline__ void load(const int32_t* p) { lo = (uint32_t)*p; }
  __device__ __forceinline__ bool whole() const { return true; }
  __device__ __forceinline__ void drop() { lo = ~0u; }
};
struct Token64 {
  uint32_t lo, hi;
  __device__ __forceinline__ void load(const int64_t* p) {
    const uint64_t v = (uint64_t)*p;
    lo = (uint32_t)v;
    hi = (uint32_t)(v >> 32);
  }
  __device__ __forceinline__ bool whole() const { return hi == 0; }
  __device__ __forceinline__ void drop() { lo = hi = ~0u; }
};
template <typename TI>
using Token = std::conditional_t<sizeof(TI) == 8, Token64, Token32>;

// Reads `run` tokens, 64 kBatch at a time, the next ones under way: f gets the
// place of the first, the tokens, the lanes whose tokens are the set's, for
// each 64, and how many those are.  under: how many tokens of the sets before.
template <typename TI, int SHIFT, bool PAD, typename F>
__device__ __forceinline__ void each_batch(const TI* __restrict__ tokens, int run, uint32_t vocab,
                                           uint32_t padding, int shift, uint32_t set,
                                           int32_t& under, const F& f) {
  const int lane = threadIdx.x & 63;
  const uint32_t mask = (1u << (SHIFT ? SHIFT : shift)) - 1;
  Token<TI> next[kBatch];
  auto fetch = [&](int i) {
    const TI* at = tokens + i;
    if (i + kList <= run) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) next[u].load(at + 64 * u + lane);
    } else {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int k = 64 * u + lane;
        next[u].load(at + (i + k < run ? k : 0));
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (i + 64 * u + lane >= run) next[u].drop();
    }
  };
  if (run > 0) fetch(0);
  for (int i = 0; i < run; i += kList) {
    uint64_t m[kBatch];
    uint32_t t[kBatch];
    int more = 0;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      t[u] = next[u].lo;
      uint64_t valid = __ballot(t[u] < vocab);
      if (sizeof(TI) == 8) valid &= __ballot(next[u].whole());
      if (PAD) valid &= ~__ballot(t[u] == padding);
      const uint32_t b = t[u] & mask;
      under += __popcll(valid & __ballot(b < set));
      m[u] = valid & __ballot(b == set);
      more += __popcll(m[u]);
    }
    if (i + kList < run) fetch(i + kList);
    if (more > 0) f(i, t, m, more);
  }
}

// Tokens of set blockIdx.x in run blockIdx.y: table[run][set][bin], and their
// sum, sums[run][set].
template <typename TI, bool PAD>
__global__ __launch_bounds__(64 * kSortWaves) void k_token_count(
    const TI* __restrict__ tokens, int64_t n, int chunk, uint32_t vocab, uint32_t padding,
    int shift, int range, int32_t* __restrict__ table, int32_t* __restrict__ sums) {
  __shared__ int32_t counts[kSplitRange], wave_total[kSortWaves];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t c0 = (int64_t)blockIdx.y * chunk;
  const int size = (int)(n - c0 < chunk ? n - c0 : chunk);
  const int share = ((size + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;
  const int left = size - w * share, run = left < 0 ? 0 : left < share ? left : share;
  for (int k = threadIdx.x; k < range; k += 64 * kSortWaves) counts[k] = 0;
  __syncthreads();
  int32_t under = 0, mine = 0;
  each_batch<TI, 0, PAD>(
      tokens + c0 + w * share, run, vocab, padding, shift, blockIdx.x, under,
      [&](int, const uint32_t(&t)[kBatch], const uint64_t(&m)[kBatch], int more) {
        mine += more;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          if (m[u] == 0) continue;
          const uint32_t b = t[u] >> shift;
          const uint32_t b0 = __builtin_amdgcn_readlane(b, __builtin_ctzll(m[u]));
          // one token many times over would meet itself in the atomics
          if ((m[u] & __ballot(b == b0)) == m[u]) {
            if (lane == 0)
              __hip_atomic_fetch_add(&counts[b0], __popcll(m[u]), __ATOMIC_RELAXED,
                                     __HIP_MEMORY_SCOPE_WORKGROUP);
          } else if (m[u] >> lane & 1) {
            __hip_atomic_fetch_add(&counts[b], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
          }
        }
      });
  if (lane == 0) wave_total[w] = mine;
  __syncthreads();
  const int64_t at = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  for (int k = threadIdx.x; k < range; k += 64 * kSortWaves) table[at * range + k] = counts[k];
  if (threadIdx.x == 0) {
    int32_t all = 0;
    for (int j = 0; j < kSortWaves; ++j) all += wave_total[j];
    sums[at] = all;
  }
}

// A run of at most kShortRun tokens has room for a token's places in 16 bits
// (the last of them may wrap to 0: nothing comes after it); longer ones (more
// than 16 kShortRun tokens in all) take 32 bits and half as many bins a block.
constexpr int kShortRun = 1 << 16;
enum Split { kOneLaunch, kRuns, kLongRuns };

template <typename TI, typename TO, int SHIFT, bool PAD, Split SPLIT>
__global__ __launch_bounds__(64 * kSortWaves) void k_token_sort(
    const TI* __restrict__ tokens, int64_t n, int chunk, uint32_t vocab, uint32_t padding,
    int shift, int range, int bits, const int32_t* __restrict__ table,
    const int32_t* __restrict__ sums, int32_t* __restrict__ order, int32_t* __restrict__ sorted,
    int32_t* __restrict__ total, TO* __restrict__ dW, int dim) {
  constexpr int RANGE = SPLIT == kOneLaunch ? kOneRange
                        : SPLIT == kRuns    ? kSplitRange
                                            : kWideRange;
  constexpr bool WIDE = SPLIT == kLongRuns;
  using Count = std::conditional_t<WIDE, uint32_t, uint16_t>;
  using lds_count = std::conditional_t<WIDE, lds_u32, lds_u16>;
  constexpr int WORDS = RANGE * (int)sizeof(Count) / 4;
  constexpr int BINS = RANGE > 64 * kSortWaves ? RANGE / (64 * kSortWaves) : 1;   // a thread
  __shared__ uint32_t counts[kSortWaves][WORDS];
  __shared__ int32_t place[RANGE];
  __shared__ uint32_t lists[kSortWaves][kList];
  __shared__ int32_t below[kSortWaves], wave_total[kSortWaves];
  __shared__ uint8_t empty[RANGE];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint64_t before = ((uint64_t)1 << lane) - 1;
  const uint32_t set = blockIdx.x;
  const int64_t c0 = (int64_t)blockIdx.y * chunk;
  const int size = (int)(n - c0 < chunk ? n - c0 : chunk);
  const int share = ((size + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;   // < 2^kRunBits
  const int left = size - w * share, run = left < 0 ? 0 : left < share ? left : share;
  const int64_t i0 = c0 + w * share;
  lds_count* count = (lds_count*)counts[w];
  lds_u32* list = (lds_u32*)lists[w];
  const int words = (range * (int)sizeof(Count) + 3) / 4;
  for (int k = lane; k < words; k += 64) counts[w][k] = 0;
  __syncthreads();

  // Counts (or, once the counts hold places, places) the first `len` listed.
  auto settle = [&](int len, bool placing) {
    for (int k = 0; k < len; k += 64) {
      const bool in = k + lane < len;
      const uint32_t entry = in ? list[k + lane] : 0;
      const int b = (int)(entry >> kRunBits);
      const uint64_t live = __ballot(in);
      const int b0 = __builtin_amdgcn_readfirstlane(b);
      uint64_t peers = live & __ballot(b == b0);
      const bool one = peers == live;       // all of them the same token
      if (!placing) {
        if (one) {
          if (lane == 0) count[b0] = (Count)(count[b0] + __popcll(live));
        } else if (in) {
          __hip_atomic_fetch_add(&counts[w][WIDE ? b : b >> 1], WIDE ? 1u : 1u << (b & 1) * 16,
                                 __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        }
        continue;
      }
      if (!one) {
        uint32_t lo = (uint32_t)live, hi = (uint32_t)(live >> 32);
        for (int d = 0; d < bits; ++d) {
          const int32_t bit = (int32_t)((uint32_t)b << (31 - d)) >> 31;
          const uint64_t v = __ballot(bit != 0);
          lo &= ~((uint32_t)v ^ bit);
          hi &= ~((uint32_t)(v >> 32) ^ bit);
        }
        peers = ((uint64_t)hi << 32) | lo;
      }
      if (in) {
        const int c = (int)count[b];
        const int32_t p = place[b] + c + __popcll(peers & before);
        order[p] = (int32_t)(i0 + (entry & ((1u << kRunBits) - 1)));
        sorted[p] = (int32_t)(((uint32_t)b << shift) + set);
        __builtin_amdgcn_wave_barrier();
        if ((peers & before) == 0) count[b] = (Count)(c + __popcll(peers));
      }
      __builtin_amdgcn_wave_barrier();
    }
  };
  // Lists the wave's part, settling full lists; returns what is still listed.
  bool whole = true;      // the list holds all of the wave's positions
  int32_t under = 0;
  auto scan = [&](bool placing) {
    int len = 0;
    each_batch<TI, SHIFT, PAD>(
        tokens + i0, run, vocab, padding, shift, set, under,
        [&](int i, const uint32_t(&t)[kBatch], const uint64_t(&m)[kBatch], int more) {
          if (len + more > kList) {
            settle(len, placing);
            whole = false;
            len = 0;
          }
#pragma unroll
          for (int u = 0; u < kBatch; ++u) {
            if (m[u] == 0) continue;
            if (m[u] >> lane & 1)
              list[len + __popcll(m[u] & before)] =
                  (t[u] >> shift) << kRunBits | (uint32_t)(i + 64 * u + lane);
            len += __popcll(m[u]);
          }
        });
    return len;
  };

  int len = scan(false);
  settle(len, false);
  if (SPLIT != kOneLaunch) {
    // tokens of the sets before this one, in all runs
    under = 0;
    for (int k = threadIdx.x; k < (int)(gridDim.x * gridDim.y); k += 64 * kSortWaves)
      under += k % gridDim.x < set ? sums[k] : 0;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) under += __shfl_xor(under, o);
  }
  if (lane == 0) below[w] = under;
  __syncthreads();
  // thread k holds the bins from k BINS on
  int32_t all[BINS], sum = 0;
#pragma unroll
  for (int q = 0; q < BINS; ++q) {
    const int k = threadIdx.x * BINS + q;
    int32_t earlier = 0;              // in the runs before this one
    all[q] = 0;
    if (k < range) {
      if (SPLIT != kOneLaunch) {
        for (int r0 = 0; r0 < (int)gridDim.y; r0 += 8) {
          int32_t c[8];
#pragma unroll
          for (int r = 0; r < 8; ++r)
            c[r] = table[((int64_t)min(r0 + r, (int)gridDim.y - 1) * gridDim.x + set) * range + k];
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            all[q] += r0 + r < (int)gridDim.y ? c[r] : 0;
            earlier += r0 + r < (int)blockIdx.y ? c[r] : 0;
          }
        }
      }
      int32_t here = 0;
#pragma unroll
      for (int j = 0; j < kSortWaves; ++j) {
        lds_count* slot = (lds_count*)counts[j] + k;
        const int c = (int)*slot;
        *slot = (Count)here;
        here += c;
      }
      if (SPLIT == kOneLaunch) all[q] = here;
      place[k] = earlier;
      empty[k] = all[q] == 0 && ((uint32_t)k << shift) + set < vocab;
    }
    sum += all[q];
  }
  int32_t incl = sum;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int32_t up = __shfl_up(incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 63) wave_total[w] = incl;
  __syncthreads();
  int32_t at = incl - sum;
  for (int j = 0; j < kSortWaves; ++j) at += below[j] + (j < w ? wave_total[j] : 0);
#pragma unroll
  for (int q = 0; q < BINS; ++q) {
    const int k = threadIdx.x * BINS + q;
    if (k < range) place[k] += at;
    at += all[q];
    if (k == range - 1 && set == gridDim.x - 1 && blockIdx.y == 0) *total = at;
  }
  __syncthreads();
  if (dW) {
    constexpr int V = 16 / (int)sizeof(TO);
    const float zero[V] = {};
    const int pieces = (dim + V - 1) / V;
    int lanes = 64;                       // threads a row
    while (lanes > 1 && lanes >= 2 * pieces) lanes >>= 1;
    const int rows = 64 / lanes;
    for (int r = (blockIdx.y * kSortWaves + w) * rows + lane / lanes; r < range;
         r += gridDim.y * kSortWaves * rows)
      if (empty[r]) {
        TO* row = dW + (((int64_t)r << shift) + set) * dim;
        for (int c = lane % lanes * V; c < dim; c += lanes * V) {
          if (c + V <= dim) store_vec<V>(row + c, zero);
          else
            for (int j = c; j < dim; ++j) put(row + j, 0.f);
        }
      }
  }
  if (!whole) len = scan(true);
  settle(len, true);
}

// ---------------------------------------------------------------------------
// Sums.  The sorted positions are cut evenly, however often a token occurs:
// `span` positions a wave, kSumWaves waves a block (and 64 V columns).  A wave
// writes the rows of the tokens that lie inside its positions.  The rows that
// a wave adds up for a token begun before it go to LDS, and the wave in which
// the token begins collects them; what a block adds up for tokens that cross
// its own borders goes to part[2 block] (begun before the block) and
// part[2 block + 1] (begun in it), and k_embed_join adds those.  Only
// neighbours in sorted[] are looked at, so nothing is loaded but order[] and
// sorted[], and then the rows.  Bound by HBM: 65536 x 768 bfloat16 into 1024
// rows takes 17 us (5.8 TB/s), 65536 x 2048 90 us with 162 MB written (4.8).
// ---------------------------------------------------------------------------
constexpr int kSumWaves = 8;

// out = scale * acc, or += where the caller accumulates.
template <int V, typename TO>
__device__ __forceinline__ void write_row(TO* out, const float (&acc)[V], int skip, float scale,
                                          int accumulate) {
  float v[V];
#pragma unroll
  for (int k = 0; k < V; ++k) v[k] = scale * acc[k];
  if (accumulate) {
    Piece<TO, V> old;
    old.load(out);
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] += old[k];
  }
  store_own<V>(out, skip, v);
}

// The sums of a block of WAVES waves, each over `have` sorted positions.  Lane
// i's tok: the token at the wave's position i - 1 (-1 outside the order), row:
// the batch position at its position i.  leave(0, sum): of a token begun before
// the block, leave(1, sum): of one begun in it that goes on after it.  ONCE: dY
// is read with the non-temporal hint.
template <int WAVES, int V, bool ONCE, typename T, typename TO, typename Leave>
__device__ __forceinline__ void sum_block(const T* __restrict__ dY, int64_t dys, int32_t tok,
                                          int32_t row, int have, const Place<V>& at, int w,
                                          float (&heads)[WAVES][64 * V], int (&through)[WAVES],
                                          TO* __restrict__ dW, int dim, float scale,
                                          int accumulate, const Leave& leave) {
  constexpr int U = 8;      // rows in flight
  const int lane = threadIdx.x & 63;
  // bit i: the token at position i is not the one before it
  const uint64_t changes = __ballot(tok != __shfl_up(tok, 1)) >> 1;
  int32_t cur = __builtin_amdgcn_readlane(tok, 1);
  bool head = have > 0 && !(changes & 1);   // the first token began before this wave
  const bool begun = head;
  float acc[V];
#pragma unroll
  for (int k = 0; k < V; ++k) acc[k] = 0.f;
  // The sum of a token that ends here, or of the first one's rows.
  auto flush = [&]() {
    if (head) store_vec<V>(&heads[w][lane * V], acc);
    else write_row<V>(dW + (int64_t)cur * dim + at.c, acc, at.skip, scale, accumulate);
    head = false;
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.f;
  };
  for (int i = 0; i < have; i += U) {
    Piece<T, V> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = __builtin_amdgcn_readlane(row, i + u < have ? i + u : i);
      v[u].template load<ONCE>(dY + r * dys + at.c);
    }
    const uint32_t turns = (uint32_t)(changes >> i) & ((1u << U) - 1) & (i == 0 ? ~1u : ~0u);
    if (turns == 0 && i + U <= have) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] += v[u][k];
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + u < have) {
          if (turns >> u & 1) {
            flush();
            cur = __builtin_amdgcn_readlane(tok, i + u + 1);
          }
#pragma unroll
          for (int k = 0; k < V; ++k) acc[k] += v[u][k];
        }
    }
  }
  // does the last token go on after this wave?
  const bool on = have > 0 && !(changes >> have & 1);
  const bool tail = on && !head;        // ... having begun in it
  if (lane == 0) through[w] = on && head;
  if (have > 0 && !tail) flush();
  __syncthreads();
  // Adds the heads of waves j.. to acc while the token goes on; whether it
  // leaves the block.
  auto collect = [&](int j) {
    for (; j < WAVES; ++j) {
      Piece<float, V> v;
      v.load(&heads[j][lane * V]);
#pragma unroll
      for (int k = 0; k < V; ++k) acc[k] += v[k];
      if (!through[j]) return false;
    }
    return true;
  };
  if (tail) {
    if (collect(w + 1)) leave(1, acc);
    else write_row<V>(dW + (int64_t)cur * dim + at.c, acc, at.skip, scale, accumulate);
  }
  if (w == 0 && begun) {
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.f;
    collect(0);
    leave(0, acc);
  }
}

template <typename T, typename TO, int V, bool ONCE>
__global__ __launch_bounds__(64 * kSumWaves) void k_embed_sum(
    const T* __restrict__ dY, int64_t dys, const int32_t* __restrict__ order,
    const int32_t* __restrict__ sorted, const int32_t* __restrict__ total, int dim, int span,
    int slices, float scale, TO* __restrict__ dW, int accumulate,
    float* __restrict__ part) {
  __shared__ float heads[kSumWaves][64 * V];
  __shared__ int through[kSumWaves];
  const int block = blockIdx.x / slices, slice = blockIdx.x - block * slices;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n = *total;
  const int64_t p0 = ((int64_t)block * kSumWaves + w) * span;
  if (p0 - w * span >= n) return;       // the whole block
  const int have = (int)(n - p0 < span ? (n > p0 ? n - p0 : 0) : span);
  const int64_t q = p0 + lane - 1;
  const int32_t tok = lane <= span + 1 && q >= 0 && q < n ? sorted[q] : -1;
  const int32_t row = lane < have ? order[p0 + lane] : 0;
  const Place<V> at((slice * 64 + lane) * V, dim);
  sum_block<kSumWaves, V, ONCE>(dY, dys, tok, row, have, at, w, heads, through, dW, dim, scale,
                                accumulate, [&](int which, const float(&acc)[V]) {
                                  store_own<V>(part + (2 * (int64_t)block + which) * dim + at.c,
                                               at.skip, acc);
                                });
}

// ---------------------------------------------------------------------------
// Small batches, in one launch: a block reads the batch, H tokens a thread,
// lists the positions of its set's tokens in order, gives each its place by
// counting the listed ones that go before it, and sums the rows from there: 16
// waves of up to kSmallSpan positions a round.  H = 1 has all in one round; with
// H = 2 what crosses from one round to the next stays in the block.  Blocks of
// the same set divide the columns (64 V each).  Bound by that chain of steps:
// 777 tokens over 1000 x 257 take 6.4 us.
// ---------------------------------------------------------------------------
constexpr int kSmallWaves = 16;
constexpr int kSmallSpan = 56;      // positions a wave, + 2 neighbours, in 64 lanes
constexpr int small_batch(int h) { return kSmallWaves * (h == 1 ? kSmallSpan : 64 * h); }

template <typename T, typename TI, typename TO, int V, int H>
__global__ __launch_bounds__(64 * kSmallWaves) void k_embed_small(
    const T* __restrict__ dY, int64_t dys, const TI* __restrict__ tokens, int n, uint32_t vocab,
    uint32_t padding, int shift, int range, float scale, TO* __restrict__ dW, int dim,
    int accumulate) {
  constexpr int W = 8, THREADS = 64 * kSmallWaves;     // W: listed tokens a step
  constexpr int kSmall = small_batch(H);
  __shared__ float heads[kSmallWaves][64 * V], crossing[2][64 * V];
  __shared__ int through[kSmallWaves], found[H * kSmallWaves];
  __shared__ uint32_t bins[kSmall + W];
  __shared__ uint16_t at_list[kSmall], order[kSmall];
  __shared__ int32_t sorted[kSmall];
  __shared__ uint8_t touched[kOneRange];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t set = blockIdx.x;
  uint32_t t[H];
  bool in[H];
  uint64_t m[H];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const int p = h * THREADS + threadIdx.x;
    t[h] = ~0u;
    in[h] = false;
    if (p < n) {
      Token<TI> token;
      token.load(tokens + p);
      t[h] = token.lo;
      in[h] = token.whole() && t[h] < vocab && t[h] != padding &&
              (t[h] & ((1u << shift) - 1)) == set;
    }
    m[h] = __ballot(in[h]);
    if (lane == 0) found[h * kSmallWaves + w] = __popcll(m[h]);
  }
  for (int k = threadIdx.x; k < range; k += THREADS) touched[k] = 0;
  __syncthreads();
  int count = 0, first[H] = {};
#pragma unroll
  for (int j = 0; j < H * kSmallWaves; ++j) {
    if (j % kSmallWaves == w) first[j / kSmallWaves] = count;
    count += found[j];
  }
#pragma unroll
  for (int h = 0; h < H; ++h)
    if (in[h]) {
      const int k = first[h] + __popcll(m[h] & (((uint64_t)1 << lane) - 1));
      bins[k] = t[h] >> shift;
      at_list[k] = (uint16_t)(h * THREADS + threadIdx.x);
      touched[t[h] >> shift] = 1;
    }
  if (threadIdx.x < W) bins[count + threadIdx.x] = ~0u;   // goes before no other
  __syncthreads();
  // a table of up to B rows, or a frequent token: nothing to sort (800 equal
  // tokens would take 60 us)
  bool same = true;
  for (int k = threadIdx.x; k < count; k += THREADS) same &= bins[k] == bins[0];
  const bool one = __syncthreads_and(same);
  for (int k = threadIdx.x; k < count; k += THREADS) {
    const uint32_t mine = bins[k];
    int place = one ? k : 0;
    if (!one)
      for (int j = 0; j < count; j += W)
#pragma unroll
        for (int u = 0; u < W; ++u) {
          const uint32_t other = bins[j + u];
          place += other < mine || (other == mine && j + u < k);
        }
    order[place] = at_list[k];
    sorted[place] = (int32_t)((mine << shift) + set);
  }
  const Place<V> at(((int)blockIdx.y * 64 + lane) * V, dim);
  if (!accumulate) {
    const float zero[V] = {};
    for (int r = w; r < range; r += kSmallWaves)
      if (!touched[r] && ((uint32_t)r << shift) + set < vocab)
        store_own<V>(dW + (((int64_t)r << shift) + set) * dim + at.c, at.skip, zero);
  }
  __syncthreads();
  const auto token = [&](int p) { return p >= 0 && p < count ? sorted[p] : -1; };
  float held[V];        // wave 0: of a token that goes on from the last round
#pragma unroll
  for (int k = 0; k < V; ++k) held[k] = 0.f;
  for (int base = 0; base < count;) {
    const int left = count - base;
    const int want = (left + 8 * kSmallWaves - 1) / (8 * kSmallWaves) * 8;
    const int span = want < kSmallSpan ? want : kSmallSpan;
    const int end = left < span * kSmallWaves ? count : base + span * kSmallWaves;
    const int p0 = base + w * span;
    const int have = end - p0 < span ? (end > p0 ? end - p0 : 0) : span;
    const int32_t tok = lane <= span + 1 ? token(p0 + lane - 1) : -1;
    const int32_t row = lane < have ? order[p0 + lane] : 0;
    sum_block<kSmallWaves, V, false>(dY, dys, tok, row, have, at, w, heads, through, dW, dim,
                                     scale, accumulate, [&](int which, const float(&acc)[V]) {
                                       store_vec<V>(&crossing[which][lane * V], acc);
                                     });
    if (H == 1) return;
    __syncthreads();
    const int32_t front = token(base), back = token(end - 1);
    const bool begun = token(base - 1) == front, on = token(end) == back;
    if (w == 0) {
      const bool all = begun && on && front == back;    // the whole round
      if (begun) {
#pragma unroll
        for (int k = 0; k < V; ++k) held[k] += crossing[0][lane * V + k];
        if (!all)
          write_row<V>(dW + (int64_t)front * dim + at.c, held, at.skip, scale, accumulate);
      }
      if (on && !all)
#pragma unroll
        for (int k = 0; k < V; ++k) held[k] = crossing[1][lane * V + k];
    }
    __syncthreads();
    base = end;
  }
}

// Adds the parts of a token that begins in block b of the sums (blockIdx.x)
// and goes on in the next, for 64 V columns: a wave each over a quarter of the
// consecutive parts.  In double: there can be thousands of parts, and their
// sum is where a float would lose most.  Bound by its launch, 4 us, where no
// token fills many blocks.
template <typename TO, int V>
__global__ __launch_bounds__(256) void k_embed_join(const float* __restrict__ part,
                                                    const int32_t* __restrict__ sorted,
                                                    const int32_t* __restrict__ total, int dim,
                                                    int positions, float scale,
                                                    TO* __restrict__ dW, int accumulate) {
  __shared__ double sh[4][64 * V];
  const int64_t b = blockIdx.x, p0 = b * positions, p1 = p0 + positions;
  const int64_t n = *total;
  if (p1 >= n) return;
  const int32_t t = sorted[p1 - 1];
  if (sorted[p1] != t || (b > 0 && sorted[p0 - 1] == t)) return;
  // the blocks after b that begin with t: equal tokens are neighbours
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int64_t more = 0;
  for (int64_t j = b + 1;; j += 64) {
    const int64_t at = (j + lane) * positions;
    const int found = __popcll(__ballot(at < n && sorted[at < n ? at : 0] == t));
    more += found;
    if (found < 64) break;
  }
  // parts: 2b + 1, then 2j for each of those
  const Place<V> at(((int)blockIdx.y * 64 + lane) * V, dim);
  const int64_t run = (more + 4) / 4;
  const int64_t j1 = (w + 1) * run < more + 1 ? (w + 1) * run : more + 1;
  double acc[V];
#pragma unroll
  for (int k = 0; k < V; ++k) acc[k] = 0.;
#pragma unroll 8
  for (int64_t j = w * run; j < j1; ++j) {
    Piece<float, V> v;
    v.load(part + (2 * (b + j) + (j == 0)) * dim + at.c);
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] += v[k];
  }
#pragma unroll
  for (int k = 0; k < V; ++k) sh[w][k * 64 + lane] = acc[k];
  __syncthreads();
  if (w > 0) return;
  float sum[V];
#pragma unroll
  for (int k = 0; k < V; ++k)
    sum[k] = (float)(((acc[k] + sh[1][k * 64 + lane]) + sh[2][k * 64 + lane]) +
                     sh[3][k * 64 + lane]);
  write_row<V>(dW + (int64_t)t * dim + at.c, sum, at.skip, scale, accumulate);
}

namespace {

constexpr int64_t kMaxBlocks = 1 << 16;   // larger grids loop

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Positions a wave of the sums.
int span_of(int64_t n) { return n <= 32768 ? 8 : n <= 131072 ? 16 : 32; }

// Blocks of the one-launch form, each of which lists the batch anew.  800
// tokens take 8.9 us instead of 16.1 (table of 30000 x 64) and 22.3 instead of
// 31.4 (50257 x 768), 1618 tokens 11.6 instead of 16.5 (53813 x 10); with more
// column slices the listing costs more than two launches (300 tokens, 300 x
// 4000: 20.2 against 15.4 us).
constexpr int64_t kSmallBlocks = 1024;

// Runs of the sort.  One launch reads the batch in every block: 65536 tokens
// over 1024 x 768 take 32 us with it and 35 in two, 40000 over 100000 x 64
// kernels of 15 and 7 + 21 us, 131072 over 3000 x 512 85 and 47 us a call.
// (One token repeated, which one block places alone: 65536 over 300 x 1024 98
// and 74 us.)  More runs than one per 16384 tokens shorten the placing where
// the table is small (131072 over 3000 x 512: 14 against 17 us for the two) and
// lengthen it where sets are many (50257 x 256: 34 against 23).
int64_t runs_of(int64_t n) {
  if (n <= 65536) return 1;
  const int64_t r = std::min<int64_t>((n + 16383) / 16384, 16);
  return std::max<int64_t>(r, (n + (1 << 19) - 1) >> 19);   // a wave's part below 2^kRunBits
}

struct GradPlan {
  int shift, range, bits, span;
  int64_t runs, chunk, sets;   // of the sort
  bool wide;                   // runs too long for 16-bit counts
  int64_t blocks;              // of the sums
  bool small;                  // one launch for all, no workspace
  size_t order, sorted, count, table, sums, part, total;
  GradPlan(int64_t n, int64_t vocab, int64_t dim) {
    runs = runs_of(n);
    chunk = runs == 1 ? n : ((n + runs - 1) / runs + 1023) / 1024 * 1024;
    // sets: about a block a CU, and no more tokens a set than it can count
    wide = chunk > kShortRun;
    const int most = runs == 1 ? kOneRange : wide ? kWideRange : kSplitRange;
    shift = kOneShift;
    while (runs > 1 && shift > 4 && (runs << (shift - 1)) >= 256) --shift;
    while ((vocab - 1) >> shift >= most) ++shift;
    range = (int)((vocab - 1) >> shift) + 1;
    for (bits = 0; (1 << bits) < range;) ++bits;
    sets = std::min<int64_t>((int64_t)1 << shift, vocab);
    span = span_of(n);
    blocks = (n + span * kSumWaves - 1) / (span * kSumWaves);
    small = n <= small_batch(2) && sets * ((dim + 255) / 256) <= kSmallBlocks;
    order = 0;
    sorted = order + align256((size_t)n * 4);
    count = sorted + align256((size_t)n * 4);
    table = count + 256;
    sums = table + (runs > 1 ? align256((size_t)runs * sets * range * 4) : 0);
    part = sums + (runs > 1 ? align256((size_t)runs * sets * 4) : 0);
    // one block has no neighbours
    total = small ? 0 : part + (blocks > 1 ? align256((size_t)blocks * 2 * dim * 4) : 0);
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
                      int32_t* total, hipStream_t s) {
  const dim3 grid((unsigned)pl.sets, (unsigned)pl.runs), block(64 * kSortWaves);
  int32_t* table = (int32_t*)((char*)a.ws + pl.table);
  int32_t* sums = (int32_t*)((char*)a.ws + pl.sums);
  const bool pad = a.padding >= 0;
  if (pl.runs > 1) {
    hipLaunchKernelGGL((pad ? k_token_count<TI, true> : k_token_count<TI, false>), grid, block, 0,
                       s, (const TI*)a.tokens, a.n, (int)pl.chunk, (uint32_t)a.vocab,
                       (uint32_t)a.padding, pl.shift, pl.range, table, sums);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const auto kernel = pl.wide ? (pad ? k_token_sort<TI, TO, 0, true, kLongRuns>
                                     : k_token_sort<TI, TO, 0, false, kLongRuns>)
                      : pl.runs > 1 ? (pad ? k_token_sort<TI, TO, 0, true, kRuns>
                                           : k_token_sort<TI, TO, 0, false, kRuns>)
                      : pl.shift == kOneShift && !pad
                          ? k_token_sort<TI, TO, kOneShift, false, kOneLaunch>
                          : k_token_sort<TI, TO, 0, true, kOneLaunch>;
  hipLaunchKernelGGL(kernel, grid, block, 0, s, (const TI*)a.tokens, a.n, (int)pl.chunk,
                     (uint32_t)a.vocab, (uint32_t)a.padding, pl.shift, pl.range, pl.bits, table,
                     sums, order, sorted, total, a.accumulate ? nullptr : (TO*)a.dW, (int)a.dim);
  return hipGetLastError();
}

template <typename T, typename TO, int V>
hipError_t embed_sum(const EmbedGradArgs& a, const GradPlan& pl, const int32_t* order,
                     const int32_t* sorted, const int32_t* total, float* part, hipStream_t s) {
  const int64_t slices = (a.dim + 64 * V - 1) / (64 * V);
  const bool once = a.n * a.dim * (int64_t)sizeof(T) + a.vocab * a.dim * (int64_t)sizeof(TO) >
                    kCacheBytes;
  hipLaunchKernelGGL((once ? k_embed_sum<T, TO, V, true> : k_embed_sum<T, TO, V, false>),
                     dim3((unsigned)(pl.blocks * slices)), dim3(64 * kSumWaves), 0, s,
                     (const T*)a.dY, a.dy_stride, order, sorted, total, (int)a.dim, pl.span,
                     (int)slices, a.scale, (TO*)a.dW, a.accumulate, part);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || pl.blocks <= 1) return e;
  hipLaunchKernelGGL((k_embed_join<TO, V>), dim3((unsigned)pl.blocks, (unsigned)slices), dim3(256),
                     0, s, part, sorted, total, (int)a.dim, pl.span * kSumWaves, a.scale,
                     (TO*)a.dW, a.accumulate);
  return hipGetLastError();
}

template <typename T, typename TI, typename TO>
hipError_t embed_small(const EmbedGradArgs& a, const GradPlan& pl, hipStream_t s) {
  const auto go = [&](auto kernel, int v) {
    const dim3 grid((unsigned)pl.sets,
                    (unsigned)((a.dim + 64 * v - 1) / (64 * v)));
    hipLaunchKernelGGL(kernel, grid, dim3(64 * kSmallWaves), 0, s, (const T*)a.dY, a.dy_stride,
                       (const TI*)a.tokens, (int)a.n, (uint32_t)a.vocab, (uint32_t)a.padding,
                       pl.shift, pl.range, a.scale, (TO*)a.dW, (int)a.dim, a.accumulate);
    return hipGetLastError();
  };
  if (a.n <= small_batch(1))
    return a.dim >= 4 ? go(k_embed_small<T, TI, TO, 4, 1>, 4)
                      : go(k_embed_small<T, TI, TO, 1, 1>, 1);
  return a.dim >= 4 ? go(k_embed_small<T, TI, TO, 4, 2>, 4)
                    : go(k_embed_small<T, TI, TO, 1, 2>, 1);
}

template <typename T, typename TO>
hipError_t embed_grad(const EmbedGradArgs& a, hipStream_t s) {
  const GradPlan pl(a.n, a.vocab, a.dim);
  if (pl.small)
    return a.token_bits == 64 ? embed_small<T, int64_t, TO>(a, pl, s)
                              : embed_small<T, int32_t, TO>(a, pl, s);
  char* ws = (char*)a.ws;
  int32_t* order = (int32_t*)(ws + pl.order);
  int32_t* sorted = (int32_t*)(ws + pl.sorted);
  int32_t* total = (int32_t*)(ws + pl.count);
  float* part = (float*)(ws + pl.part);
  hipError_t e = a.token_bits == 64 ? token_sort<int64_t, TO>(a, pl, order, sorted, total, s)
                                    : token_sort<int32_t, TO>(a, pl, order, sorted, total, s);
  if (e != hipSuccess || a.n == 0) return e;
  return a.dim >= 4 ? embed_sum<T, TO, 4>(a, pl, order, sorted, total, part, s)
                    : embed_sum<T, TO, 1>(a, pl, order, sorted, total, part, s);
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
