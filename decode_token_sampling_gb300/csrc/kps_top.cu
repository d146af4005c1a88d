// kps_top.cu — the top logits of every row with the log-sum-exps that turn them into
// log-probabilities: what serving returns beside a sampled token, and what a teacher hands to
// the distillation loss.
//
// Per row, with the order "value descending, index ascending" (NaN counts as -inf) and a = x / tau:
//
//   ids, values = the first n elements of the order       lse  = ln sum_v exp(a_v)
//   rest = ln sum_{v not among them} exp(a_v)             logprob = a_token - lse
//
// One pass over the row, at best as fast as memory delivers it.  A threshold from a sample of
// the row is reached by a few times n elements.  A 16-byte vector holding one of those goes to a
// list in shared memory whole (one ballot and two stores; taking single elements out of the
// vector cost four times the instructions of the sum itself), all others into a running sum of
// exponentials.  Then digits of the listed keys, counted, cut the list to little more than n
// elements, which the first digit's counts also put in order but for the few that share one: these
// are ranked pairwise.  Everything else in the list joins the sum.  So the rest is a sum of
// its own, never a difference of two large ones.  A list that came out too short or too long (the
// sample misjudged the row, or ties crowd the threshold) sends the row to an exact selection.
//
// 2048 rows of 151936 bf16: 121 us (92 at the copy rate); warps issue on 47% of the cycles, waiting
// for loads first (an SM's four rows are not always at different phases).  256 rows of them: 21 us
// (11.5), where the sample's threshold and the list's selection have too few rows behind them to
// hide in; one row of 151936 fp32: 9.8 us, a chain of latencies.  The sample's size sets the list's:
// one element in 37 of a row looked at left 550 vectors of 19000 in the list of the top 64 and the
// pass bound by its instructions, 137 us; one in nine, read as whole vectors, 121.
// Measured slower: the next round's loads issued before this one's sums (125-130 us).

#include "kps.h"
#include "kps_host.h"
#include "kps_stream.cuh"

#include <cooperative_groups.h>

#include <climits>
#include <cmath>
#include <type_traits>

namespace cg = cooperative_groups;

namespace kps {
namespace top {

using namespace stream;

constexpr int kNT = 256;  // threads per CTA
constexpr int kNW = kNT / 32;
// 16-byte loads each thread keeps in flight.  Six with four CTAs an SM (64 registers) took 121 us
// for 2048 rows of 151936 bf16 and 21.3 us for 256; five with five CTAs 118 and 22.4 us, four with
// five 3% and 8% more than that, eight with four 1% more than six on both.
constexpr int kU = 6;
constexpr int kMaxN = 1024;    // the framework's top-k limit
constexpr int64_t kMaxV = 1 << 20;
constexpr int kMaxCS = 8;      // widest cluster (the portable limit)
constexpr int kAllV = 4096;    // rows this short are listed whole
constexpr int kMaxPer = 8;     // sampled vectors per thread, at most (of a quarter million elements)
constexpr int kMaxRank = 96;   // rank of the threshold among the threads' sample maxima, at most
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;

// Capacities: listed vectors (an equal segment for each warp that reads the row) and ranked
// survivors.  The small form lets four CTAs share an SM with room left for their loads in flight
// (lines of the first-level cache); the top 128 of a long row list about 550 vectors.
constexpr int kSmallN = 128;
template <bool kSmall>
struct Caps {
  static constexpr int list = kSmall ? 1536 : 4096;
  static constexpr int words = kSmall ? 512 : 2048;
};

struct Params {
  const void* x;
  int64_t B, ld;
  int V, n;
  float tau, c;  // c = log2(e) / tau
  const int64_t* tokens;  // or nullptr
  int32_t* ids;
  float* values;
  float* lse;      // or nullptr
  float* rest;     // or nullptr
  float* logprob;  // or nullptr
};

// Keys order as the values do (-0 first made +0); an element's word orders by (value desc, index asc).
__device__ __forceinline__ uint32_t fkey(float x) {
  const uint32_t u = __float_as_uint(x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float kfloat(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
__device__ __forceinline__ float clean(float x) { return isnan(x) ? -INFINITY : x + 0.0f; }
__device__ __forceinline__ unsigned long long word_of(uint32_t key, int v) {
  return (static_cast<unsigned long long>(key) << 32) | static_cast<uint32_t>(~static_cast<uint32_t>(v));
}
__device__ __forceinline__ float word_value(unsigned long long w) { return kfloat(static_cast<uint32_t>(w >> 32)); }
__device__ __forceinline__ int word_index(unsigned long long w) { return static_cast<int>(~static_cast<uint32_t>(w)); }

template <bool kSmall>
struct Smem {
  unsigned long long words[Caps<kSmall>::words];  // the survivors
  uint4 vec[Caps<kSmall>::list];                  // the listed vectors, by warp
  int32_t at[Caps<kSmall>::list];                 // index of each one's first element (~: its only one)
  uint32_t hist[256];
  uint32_t offset[256], filled[256];  // by first digit: survivors with a larger one, and with it
  float red[kNW][4];
  float part[kMaxCS * kNW];    // the sums of the cluster's warps
  uint32_t seg[kMaxCS * kNW];  // vectors each warp listed
  uint32_t top_key;            // of the listed elements
  uint32_t n_words;
  uint32_t bin, above, inside;
};

// Two sums merged over the block; every thread gets the results.
__device__ __forceinline__ void block_merge2(Sum2& a, Sum2& b, float c, float (*red)[4]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  a = warp_merge(a, c);
  b = warp_merge(b, c);
  __syncthreads();
  if (lane == 0) {
    red[warp][0] = a.ref;
    red[warp][1] = a.s;
    red[warp][2] = b.ref;
    red[warp][3] = b.s;
  }
  __syncthreads();
  const float* r = red[lane & (kNW - 1)];
  a = warp_merge(Sum2{r[0], lane < kNW ? r[1] : 0.0f}, c);
  b = warp_merge(Sum2{r[2], lane < kNW ? r[3] : 0.0f}, c);
}
__device__ __forceinline__ void add_one(Sum2& sum, float x, float c) {
  if ((x - sum.ref) * c > kRaise) sum.raise(clamp_ref(x), c);
  sum.s += ex2((x - sum.ref) * c);
}

// Finds in hist (256 counts) the bin, from the top, where the running count reaches need:
// sm.bin, sm.above (the count over it) and sm.inside (its own).  With offsets, also every bin's
// count over it.  Starts and ends with a barrier.
template <class S>
__device__ __forceinline__ void find_bin(S& sm, uint32_t need, bool offsets = false) {
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    uint32_t n[8], sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      n[i] = sm.hist[255 - 8 * lane - i];
      sum += n[i];
    }
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    uint32_t acc = incl - sum;
    if (offsets) {
      uint32_t o = acc;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sm.offset[255 - 8 * lane - i] = o;
        o += n[i];
      }
    }
    if (acc < need && need <= incl) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (acc < need && need <= acc + n[i]) {
          sm.bin = 255 - 8 * lane - i;
          sm.above = acc;
          sm.inside = n[i];
        }
        acc += n[i];
      }
    }
  }
  __syncthreads();
}

// Element e of a vector as fp32.
template <bool kBF16>
__device__ __forceinline__ float elem(const uint4& w, int e) {
  const uint32_t word[4] = {w.x, w.y, w.z, w.w};
  if (kBF16) return __uint_as_float((e & 1) ? (word[e / 2] & 0xFFFF0000u) : (word[e / 2] << 16));
  return __uint_as_float(word[e]);
}

// Every element of the row, with the warp converged: f(valid, value with NaN -> -inf, index).
template <bool kBF16, class F>
__device__ __forceinline__ void each(const RowView<kBF16>& x, F&& f) {
  constexpr int G = kBF16 ? 8 : 4;
  for (int base = 0; base < x.nv; base += kNT * kU) {
    uint4 w[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int g = base + u * kNT + static_cast<int>(threadIdx.x);
      w[u] = g < x.nv ? ld_stream(x.vec + g) : neg_inf_vec<kBF16>();
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int g = base + u * kNT + static_cast<int>(threadIdx.x);
#pragma unroll
      for (int e = 0; e < G; ++e) f(g < x.nv, clean(elem<kBF16>(w[u], e)), x.head + g * G + e);
    }
  }
  const bool in = static_cast<int>(threadIdx.x) < x.loose();
  const int v = in ? x.loose_at(threadIdx.x) : 0;
  f(in, in ? clean(x.at(v)) : -INFINITY, v);
}

// The exact selection, by one CTA, for rows whose list came out too short or too long: the n-th
// element of the order by 8-bit digits of its key and, among equal keys, of its index; then the n
// elements as survivors and the thread's sum of all others.  At least n elements have a key of
// floor or more.
template <bool kBF16, class S>
__device__ __noinline__ Sum2 exact_select(const RowView<kBF16>& x, int n, uint32_t floor, float c, S& sm) {
  uint32_t need = static_cast<uint32_t>(n);
  unsigned long long at = 0;  // the digits found so far, from the top of the 64-bit word
  __syncthreads();            // everything before is done with what is written below
  if (n > 0) {
    for (int shift = 56; shift >= 0; shift -= 8) {
      if (kBF16 && shift == 40) {  // a bf16 key's low half follows from its sign
        at |= (at >> 63) ? 0ull : 0xFFFFull << 32;
        shift = 32;
        if (sm.inside == need) break;
        continue;
      }
      if (shift == 24) {  // indexes are below 2^20: the top 8 bits of their complements are ones
        at |= 0xFFull << 24;
        continue;
      }
      for (int i = threadIdx.x; i < 256; i += kNT) sm.hist[i] = 0u;
      __syncthreads();
      each<kBF16>(x, [&](bool valid, float y, int v) {
        const unsigned long long w = word_of(fkey(y), v);
        const bool ok = valid && (w >> 32) >= floor && (shift == 56 || (w >> (shift + 8)) == (at >> (shift + 8)));
        const int d = static_cast<int>((w >> shift) & 255u);
        const unsigned who = __ballot_sync(0xffffffffu, ok);
        if (who == 0u) return;
        // one add for a warp that agrees (equal values side by side would otherwise queue up)
        const int d0 = __shfl_sync(0xffffffffu, d, __ffs(who) - 1);
        if (__all_sync(0xffffffffu, !ok || d == d0)) {
          if ((threadIdx.x & 31) == 0) atomicAdd(&sm.hist[d0], static_cast<uint32_t>(__popc(who)));
        } else if (ok) {
          atomicAdd(&sm.hist[d], 1u);
        }
      });
      find_bin(sm, need);
      at |= static_cast<unsigned long long>(sm.bin) << shift;
      need -= sm.above;
      if (shift == 32 && sm.inside == need) break;  // every element equal to the n-th belongs
      __syncthreads();
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) sm.n_words = 0u;
  __syncthreads();
  Sum2 sum{-FLT_MAX, 0.0f};
  each<kBF16>(x, [&](bool valid, float y, int v) {
    const unsigned long long w = word_of(fkey(y), v);
    if (valid && n > 0 && w >= at) {
      sm.words[atomicAdd(&sm.n_words, 1u)] = w;  // n of them
    } else if (valid) {
      add_one(sum, y, c);
    }
  });
  return sum;
}

template <bool kBF16, bool kSmall>
__global__ void __launch_bounds__(kNT, kSmall ? 4 : 2) top_kernel(const Params P) {
  constexpr int G = kBF16 ? 8 : 4;
  constexpr int kWords = Caps<kSmall>::words;
  extern __shared__ __align__(16) unsigned char smem[];
  Smem<kSmall>& sm = *reinterpret_cast<Smem<kSmall>*>(smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned lt = (1u << lane) - 1u;
  const int CS = static_cast<int>(cg::this_cluster().num_blocks());
  const int rank = static_cast<int>(cg::this_cluster().block_rank());
  const int64_t row = blockIdx.x / CS;
  const int n = P.n;
  const float c = P.c;
  const RowView<kBF16> x(P.x, row * P.ld, P.V);
  const int g0 = static_cast<int>(static_cast<int64_t>(x.nv) * rank / CS);
  const int g1 = static_cast<int>(static_cast<int64_t>(x.nv) * (rank + 1) / CS);
  float token_logit = -INFINITY;
  if (threadIdx.x == 0) {
    sm.top_key = 0u;
    sm.n_words = 0u;
  }
  // every CTA of the cluster runs, and has set these, before any writes into another's shared memory
  if (CS > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  if (threadIdx.x == 0) {
    if (P.logprob && rank == 0) {
      const int64_t t = P.tokens[row];
      token_logit = t >= 0 && t < P.V ? clean(x.at(static_cast<int>(t))) : NAN;  // NaN: no such token
    }
  }

  // ---- the threshold: every CTA of the row takes the same sample --------------------------
  float thr = n > 0 ? -INFINITY : INFINITY;  // n == 0: only +inf is listed
  float ref = 0.0f;                          // of the sum: the threshold; n == 0: the largest of the sample
  if (P.V > kAllV || n == 0) {
    // kNT * per vectors (m times as many for the longest rows) in runs of eight consecutive ones, 128
    // bytes, spread over the row, and a maximum of its own for each thread.  (Longer runs see too
    // much of one place: vocabularies are ordered, and neighbours are likely alike.  Runs of four
    // took 125 us for 2048 rows of 151936 bf16, of eight 121.)  One element of the row in `one` is
    // looked at, so of the row's first n about n / one are: fewer than `want` but for one row in
    // 10^5 (a Poisson tail), so the want-th largest maximum is at most the n-th largest of the row.
    const int m = (P.V + (1 << 18) - 1) >> 18;
    int per = P.V > kAllV ? kMaxPer : 1;
    float one, r;
    for (;; per >>= 1) {
      one = fmaxf(1.0f, static_cast<float>(P.V) / static_cast<float>(kNT * G * per * m));
      r = static_cast<float>(n) / one;
      r += 4.0f * sqrtf(r) + 3.5f;
      if ((r <= static_cast<float>(kMaxRank) && kNT * G * per * m <= P.V) || per == 1) break;
    }
    constexpr int kRun = 8;
    const int step = x.nv >= kRun * m ? (x.nv - kRun * m) / (kNT / kRun * per - 1) : 0;
    float y = -INFINITY;
    for (int j = 0; j < m; ++j) {
      uint4 place[kMaxPer];  // all loads in flight together
#pragma unroll
      for (int i = 0; i < kMaxPer; ++i) {
        const int v = i * kNT + static_cast<int>(threadIdx.x);
        const int g = v / kRun * step + v % kRun + kRun * j;
        place[i] = i < per && g < x.nv ? x.vec[g] : neg_inf_vec<kBF16>();
      }
#pragma unroll
      for (int i = 0; i < kMaxPer; ++i) y = fmaxf(y, vec_max<kBF16>(place[i]));  // NaN is ignored
    }
    const uint32_t key = fkey(y + 0.0f);
    const int want = n > 0 ? static_cast<int>(r) : 1;
    uint32_t t = 0;  // the largest key, its low 16 bits zero, that `want` maxima reach
    int reach = kNT;
    for (int bit = 31; bit >= 16; --bit) {
      const uint32_t mid = t | (1u << bit);
      const int k = __syncthreads_count(key >= mid);
      if (k >= want) {
        t = mid;
        reach = k;
      }
    }
    // half of the sample shares the threshold's digits: a mask's value, as in a row that allows
    // some tokens only.  What the row can offer lies above it (if not, the list is too short).
    if (n > 0 && reach >= kNT / 2 && t > kKeyNegInf && t < 0xFF000000u) t += 0x10000u;
    if (t > kKeyNegInf) {
      ref = kfloat(t);
      if (n > 0) thr = ref;
      if (fabsf(ref * c) > kFastRef) ref = 0.0f;  // far below zero: what is not listed weighs nothing against it
    } else if (n > 0) {
      thr = -FLT_MAX;  // a row of -inf but for a few: everything finite
    }
  }
  __syncthreads();
  if (CS > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");

  // ---- the pass -----------------------------------------------------------------------------
  // everything summed here is below the threshold, the sum's reference
  FastSum<kBF16> fast(ref, c);
  // the list lives with rank 0: every warp of the cluster writes to a segment of its own there
  cg::cluster_group cl = cg::this_cluster();
  Smem<kSmall>& home = CS > 1 ? *cl.map_shared_rank(&sm, 0) : sm;
  const uint32_t seg_cap = static_cast<uint32_t>(Caps<kSmall>::list / (kNW * CS));
  const int seg = rank * kNW + warp;
  uint32_t listed = 0;  // this warp's
  uint4* const seg_vec = home.vec + seg * seg_cap;
  int32_t* const seg_at = home.at + seg * seg_cap;
  float mx = -INFINITY;  // of the listed vectors
  auto list = [&](bool hit, const uint4& w, int first, float m) {
    const unsigned who = __ballot_sync(0xffffffffu, hit);
    const uint32_t pos = listed + __popc(who & lt);
    if (hit) {
      if (pos < seg_cap) {
        seg_vec[pos] = w;
        seg_at[pos] = first;
      }
      mx = fmaxf(mx, m);
    }
    listed += __popc(who);
  };
  // a round of loads; only the last one has to look where the CTA's part ends
  auto round = [&](int base, auto full) {
    constexpr bool kFull = decltype(full)::value;
    uint4 w[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int g = base + u * kNT + static_cast<int>(threadIdx.x);
      w[u] = kFull || g < g1 ? ld_stream(x.vec + g) : neg_inf_vec<kBF16>();
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int g = base + u * kNT + static_cast<int>(threadIdx.x);
      const float m = vec_max<kBF16>(w[u]);
      const bool hit = m >= thr && (kFull || g < g1);
      if (__any_sync(0xffffffffu, hit)) {
        list(hit, w[u], x.head + g * G, m);
        if (hit) w[u] = neg_inf_vec<kBF16>();
      }
      fast.add(w[u]);
    }
  };
  int base = g0;
#pragma unroll 1
  for (; base + kNT * kU <= g1; base += kNT * kU) round(base, std::true_type{});
  if (base < g1) round(base, std::false_type{});
  Sum2 sum{ref, fast.total(ref, c)};  // one reference for all of them
  // the elements outside the vectors, each as the first of a vector of its own (its index
  // complemented): the head with rank 0, the tail with the last rank
  if (warp == 0) {
    const bool in = lane < x.loose() && ((x.loose_at(lane) < x.head) ? rank == 0 : rank == CS - 1);
    const float y = in ? x.at(x.loose_at(lane)) : -INFINITY;
    const bool hit = in && y >= thr;
    uint4 w = neg_inf_vec<kBF16>();
    w.x = kBF16 ? (0xFF800000u | (__float_as_uint(y) >> 16)) : __float_as_uint(y);
    list(hit, w, ~x.loose_at(lane), y);
    if (in && !hit) sum.s += ex2((y - ref) * c);
  }
  {
    const uint32_t k = __reduce_max_sync(0xffffffffu, fkey(mx + 0.0f));
    if (lane == 0) {
      home.seg[seg] = listed;
      atomicMax(&home.top_key, k);
    }
  }
  if (CS > 1) {
    const float s = warp_sum(sum.s);
    if (lane == 0) home.part[seg] = s;
  }
  for (int i = threadIdx.x; i < 256; i += kNT) {
    sm.hist[i] = 0u;
    sm.filled[i] = 0u;
  }
  if (CS > 1) {
    cl.sync();  // rank 0 holds everything
    if (rank != 0) return;
    sum.s = static_cast<int>(threadIdx.x) < kNW * CS ? sm.part[threadIdx.x] : 0.0f;
  } else {
    __syncthreads();
  }
  // every finite element is listed (short rows, and long ones with few finite elements): the pass
  // summed nothing, and what joins from the list may lie anywhere, far below zero too
  if (thr <= -FLT_MAX && sum.s == 0.0f) sum.ref = -FLT_MAX;  // (a NaN in the sum stays)

  // ---- the listed elements: cut to the n-th largest key's digit --------------------------------
  const int nseg = kNW * CS;
  const uint32_t most = static_cast<int>(threadIdx.x) < nseg ? sm.seg[threadIdx.x] : 0u;
  // a list that overflowed, a NaN, a sum past fp32's range: the exact selection.  A sum that
  // nothing near its reference holds up is taken again against what there is.
  const bool over = __syncthreads_or(most > seg_cap);
  const bool bad = over || !(sum.s < 0x1p100f);
  bool exact = __syncthreads_or(bad);
  const bool weak = !__syncthreads_or(sum.s >= 0x1p-60f) && thr > -FLT_MAX;
  uint32_t cut = 0xFFFFFFFFu;  // keys from here on survive
  int count = 0, digit = 0;    // the survivors, and the shift of their first digit
  const uint32_t tkey = thr == -INFINITY ? kKeyNegInf : fkey(thr + 0.0f);
  auto vectors = [&](auto&& f) {  // f(vector, index of its first element, elements) for the listed ones
    // a warp for each segment, or for as many of a cluster's shorter ones as it has CTAs (at most four)
    const int each = CS < 4 ? CS : 4, wide = 32 / each;
    for (int q = warp * each + lane / wide; q < nseg; q += kNW * each) {
      const uint32_t count = sm.seg[q];
      for (uint32_t i = lane & (wide - 1); i < count; i += wide) {
        const int v0 = sm.at[q * seg_cap + i];
        f(sm.vec[q * seg_cap + i], v0 < 0 ? ~v0 : v0, v0 < 0 ? 1 : G);
      }
    }
  };
  if (!exact && n > 0) {
    uint32_t lo = tkey, hi = sm.top_key, need = static_cast<uint32_t>(n), above = 0;
    for (bool first = true;; first = false) {
      const uint32_t span = hi - lo;
      const int shift = span >> 8 ? 24 - __clz(span) : 0;  // 256 bins over [lo, hi]
      if (first) digit = shift;
      vectors([&](const uint4& w, int, int elems) {
#pragma unroll
        for (int e = 0; e < G; ++e) {
          const uint32_t k = fkey(clean(elem<kBF16>(w, e)));
          if (k >= lo && k <= hi && e < elems) atomicAdd(&sm.hist[(k - lo) >> shift], 1u);
        }
      });
      if (threadIdx.x == 0) sm.bin = ~0u;
      find_bin(sm, need, first);
      if (sm.bin == ~0u) {  // fewer than n listed elements
        exact = true;
        break;
      }
      above += sm.above;
      need -= sm.above;
      lo += sm.bin << shift;
      const uint32_t inside = sm.inside;
      if (above + inside <= static_cast<uint32_t>(kWords)) {
        cut = lo;
        count = static_cast<int>(above + inside);
        break;
      }
      if (shift == 0) {  // more equal keys than there is room for
        exact = true;
        break;
      }
      hi = lo + (1u << shift) - 1u;
      __syncthreads();
      for (int i = threadIdx.x; i < 256; i += kNT) sm.hist[i] = 0u;
      __syncthreads();
    }
  }
  if (exact) {
    // (an overflown segment holds more than its capacity of vectors that reach the threshold)
    sum = exact_select<kBF16>(x, n, over && seg_cap >= static_cast<uint32_t>(n) ? tkey : 0u, c, sm);
    count = n;
  } else {
    vectors([&](const uint4& w, int v0, int elems) {
      float y[G];
      float m = -INFINITY;
#pragma unroll
      for (int e = 0; e < G; ++e) {
        y[e] = clean(elem<kBF16>(w, e));
        const uint32_t k = fkey(y[e]);
        if (k >= cut && e < elems) {
          const uint32_t d = (k - tkey) >> digit;
          sm.words[sm.offset[d] + atomicAdd(&sm.filled[d], 1u)] = word_of(k, v0 + e);
          y[e] = -INFINITY;
        }
        m = fmaxf(m, y[e]);
      }
      if ((m - sum.ref) * c > kRaise) sum.raise(clamp_ref(m), c);
#pragma unroll
      for (int e = 0; e < G; ++e) sum.s += ex2((y[e] - sum.ref) * c);
    });
    if (weak) {
      sum = Sum2{-FLT_MAX, 0.0f};
      each<kBF16>(x, [&](bool valid, float y, int) {
        if (valid && fkey(y) < cut) add_one(sum, y, c);
      });
    }
  }
  __syncthreads();

  // ---- ranks and outputs ------------------------------------------------------------------------
  unsigned long long* sorted = reinterpret_cast<unsigned long long*>(sm.vec);  // the list is done with
  static_assert(sizeof(sm.vec) >= sizeof(sm.words), "the survivors in order take the list's place");
  for (int i = threadIdx.x; i < count; i += kNT) {
    const unsigned long long w = sm.words[i];
    int first = 0, end = count;  // those that share the first digit
    if (!exact) {
      const uint32_t d = (static_cast<uint32_t>(w >> 32) - tkey) >> digit;
      first = static_cast<int>(sm.offset[d]);
      end = first + static_cast<int>(sm.filled[d]);
    }
    int r = first;
    for (int j = first; j < end; ++j) r += sm.words[j] > w ? 1 : 0;
    sorted[r] = w;
  }
  __syncthreads();
  Sum2 lead{-FLT_MAX, 0.0f};
  for (int i = threadIdx.x; i < count; i += kNT) {
    const unsigned long long w = sorted[i];
    const float y = word_value(w);
    if (i < n) {
      P.ids[row * n + i] = word_index(w);
      P.values[row * n + i] = y;
      add_one(lead, y, c);
    } else {
      add_one(sum, y, c);
    }
  }
  block_merge2(sum, lead, c, sm.red);
  if (threadIdx.x == 0) {
    const Sum2 all = merge(lead, sum, c);
    // a sum of nothing is -inf; a sum with +inf in it is +inf
    auto ln = [&](const Sum2& s) { return s.s == 0.0f ? -INFINITY : logf(s.s) + s.ref / P.tau; };
    const float lse = ln(all);
    if (P.lse) P.lse[row] = lse;
    if (P.rest) P.rest[row] = ln(sum);
    if (P.logprob) {
      // relative to the sum's reference: lse and the token's logit are both large, and lse may have
      // left fp32 where their difference has not (the type's lowest value over tau < 1)
      const float y = token_logit;
      float lp = all.s > 0.0f && all.s < INFINITY ? (y - all.ref) / P.tau - logf(all.s) : y / P.tau - lse;
      if (isnan(y)) lp = -INFINITY;
      P.logprob[row] = lp;
    }
  }
}

// ------------------------------------------------------------------------------------------
// Host side
// ------------------------------------------------------------------------------------------
template <bool kBF16, bool kSmall>
static kps_status launch_t(const Params& P, cudaStream_t stream) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      (sizeof(Smem<kSmall>) > 48 * 1024 &&
       cudaFuncSetAttribute(top_kernel<kBF16, kSmall>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Smem<kSmall>)) !=
           cudaSuccess)) {
    (void)cudaGetLastError();
    return KPS_ERR_CUDA;
  }
  // few rows: a cluster shares each, as wide as leaves every CTA a full round of loads
  int cs = 1;
  const int64_t round = static_cast<int64_t>(kNT) * kU * (kBF16 ? 8 : 4);
  while (cs < kMaxCS && P.B * cs * 2 <= 2 * sms && P.V >= 2 * cs * round) cs *= 2;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(static_cast<unsigned>(P.B * cs));
  lc.blockDim = dim3(kNT);
  lc.dynamicSmemBytes = sizeof(Smem<kSmall>);
  lc.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  if (cudaLaunchKernelEx(&lc, top_kernel<kBF16, kSmall>, P) != cudaSuccess) {
    (void)cudaGetLastError();
    return KPS_ERR_CUDA;
  }
  return KPS_OK;
}
template <bool kBF16>
static kps_status launch(const Params& P, cudaStream_t stream) {
  return P.n <= kSmallN ? launch_t<kBF16, true>(P, stream) : launch_t<kBF16, false>(P, stream);
}

}  // namespace top
}  // namespace kps

extern "C" kps_status kps_top_logits(const void* logits, kps_dtype dt, int64_t B, int64_t V, int64_t ld, int64_t n,
                                     float temperature, const int64_t* tokens, int32_t* out_ids, float* out_values,
                                     float* out_lse, float* out_rest, float* out_logprob, cudaStream_t stream) {
  namespace kt = kps::top;
  const kps::NvtxRange range("kps_top_logits");
  if (dt != KPS_F32 && dt != KPS_BF16) return KPS_ERR_INVALID_ARG;
  if (B < 0 || V < 1 || n < 0 || n > kt::kMaxN || n > V || (B > 1 && ld < V)) return KPS_ERR_INVALID_ARG;
  if (!(temperature > 0.0f) || std::isinf(temperature) || std::isinf(kps::stream::kLog2e / temperature)) return KPS_ERR_INVALID_ARG;
  if (V > kt::kMaxV || B > INT32_MAX / kt::kMaxCS) return KPS_ERR_UNSUPPORTED;
  if (B == 0) return KPS_OK;
  if (!logits || (n > 0 && (!out_ids || !out_values)) || (out_logprob && !tokens)) return KPS_ERR_INVALID_ARG;
  auto off = [](const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; };
  if (off(logits, dt == KPS_BF16 ? 2 : 4) || off(tokens, 8) || off(out_ids, 4) || off(out_values, 4) || off(out_lse, 4) ||
      off(out_rest, 4) || off(out_logprob, 4))
    return KPS_ERR_INVALID_ARG;
  kt::Params P = {};
  P.x = logits;
  P.B = B;
  P.ld = ld;
  P.V = static_cast<int>(V);
  P.n = static_cast<int>(n);
  P.tau = temperature;
  P.c = kps::stream::kLog2e / temperature;
  P.tokens = tokens;
  P.ids = out_ids;
  P.values = out_values;
  P.lse = out_lse;
  P.rest = out_rest;
  P.logprob = out_logprob;
  return dt == KPS_BF16 ? kt::launch<true>(P, stream) : kt::launch<false>(P, stream);
}
