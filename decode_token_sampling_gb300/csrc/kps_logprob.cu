// kps_logprob.cu — the log-probabilities of given tokens with their ranks and the entropies of their
// rows, the gradient of both, and the clipped policy loss with its gradient.
//
// The formulas are in kps_score.cuh.  With g and h the gradients of a row's log-probability and entropy:
//
//   d / d x_v = (g (delta_tv - p_v) - h p_v (d_v + Q)) / T
//
// and for the policy loss, r = exp(logprob - old), A the advantage, u = ref - logprob:
//
//   loss = w (-min(r A, clip(r, 1 - lo, 1 + hi) A) + kl (exp(u) - u - 1) - ent entropy)
//   g = w (-A r [not clipped] - kl (exp(u) - 1)),  h = -w ent
//
// All of it is bound by memory: a row is read (V elements), and written for a gradient.

#include "kps.h"
#include "kps_host.h"
#include "kps_score.cuh"
#include "kps_select.cuh"

#include <cooperative_groups.h>

#include <atomic>
#include <climits>
#include <cmath>
#include <type_traits>

namespace cg = cooperative_groups;

namespace kps {
namespace score {

using namespace select;

constexpr int kMaxCS = 8;  // widest cluster (the portable limit)

// The warp's largest value (NaN as -inf).
__device__ __forceinline__ float warp_top(float x) { return kfloat(__reduce_max_sync(0xffffffffu, fkey(no_nan(x) + 0.0f))); }

// ------------------------------------------------------------------------------------------
// Scoring with none or few alternatives: one pass
// ------------------------------------------------------------------------------------------
//
// A warp's sums are against the largest logit that it has seen, looked for once in a round of loads:
// it rises some three times in a row's dozen rounds.  The element that holds it stays out of the sums
// until a larger one takes its place.
//
// Alternatives, up to 32 of them: each thread keeps the round of its vectors that holds its largest value, in
// shared memory, and the largest value of its other rounds.  Of the threads' largest values 32, the first few of
// each warp, are put in order: the n-th of them bounds the n-th of the block's part of the row from below.  What reaches it
// lies in the kept rounds, or (the other value reaches it too: a thread in some rows) in vectors that are
// read once more: little more than n elements, ranked pairwise.  2048 rows of 128256 bf16 take 106 us with five
// alternatives, 109 with twenty, 88 without (79 at the copy rate): a block's end takes some 7 us, the last sums and
// the ranking in a chain that five blocks an SM do not hide.  The 48 registers that these leave a thread do not hold the
// pass with the kept round: 20 to 28 bytes a thread are stored to local memory and 52 to 60 loaded, up to 44 and 92 in
// first_equal, which few rows call (blocks of 512 threads have 64 registers and keep all there).  Slower (when it took
// 111 and 112): every vector above a rising bound listed during the pass (139), the kept round read again instead of kept
// (118 and 127), all vectors of those threads read again (108 and 147), the largest vector of each of a thread's five
// streams kept (131).
//
// 4096 rows of 151936 bf16, a quarter of them empty, without alternatives: 147 us (140 at the copy rate) with
// five loads in flight and five CTAs an SM; six and four 153, four and five 151, eight and four 153, eight and
// three 165; four and six 147, but 16.4 instead of 15.0 us for 333 rows of 50001 fp32, whose CTAs are few
// (13.4 with the first round fetched ahead).
// Rounds that all look where the row ends took 160 with six and four.  Blocks that go on to rows of blocks not yet
// started (cluster launch control), their warps independent of each other: 165, for the registers that it takes and
// the wait for the next row's number behind empty ones.
// 16-byte loads each thread keeps in flight (of 512 threads four: the kept rounds fit 48 KB), and the widest cluster
// of blocks of NT threads.
template <int NT>
constexpr int kLoads = NT == 512 ? 4 : 5;
template <int NT>
constexpr int kWidest = NT == 256 ? kMaxCS : 1;
// The alternatives that the kept rounds do for; more go to the top logits' kernel.  2048 rows of 128256 bf16: 32 take 124
// us, 33 there 133, 64 140, 128 149, 129 (its larger lists, two CTAs an SM instead of four) 201, 256 221, 1000 302; 256
// rows of 151936 bf16 29, 32, 34 with 32, 33, 64, and 38 with 256.
constexpr int kFew = 32;
constexpr int kWords = 512;  // elements that are ranked
template <bool kList, int NT>
struct Few {
  static constexpr int kU = kLoads<NT>;
  unsigned long long words[kWords + kFew];
  unsigned long long lists[kWidest<NT>][kFew];  // rank 0's: what each CTA found
  unsigned long long best[kFew];
  uint32_t sizes[kMaxCS];                  // and how many; ~0: more than there is room for
  uint32_t tops[kFew];                     // the keys of some threads' largest values of each warp
  uint4 kept[kU][NT];                     // each thread's round of vectors
  int32_t at[NT];                         // and its first vector
  uint16_t who[2][NT];                    // the threads whose kept vectors count, and those whose all are read again
  uint32_t n_who[2], ties[NT / 32];
  uint32_t hist[256], bin, above, inside, n_words;  // for the exact selection
  uint32_t* offset;                                 // (not asked for)
};
template <int NT>
struct Few<false, NT> {};

// The warp's keys in descending order.
__device__ __forceinline__ uint32_t sort_warp(uint32_t k) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
    for (int j = size >> 1; j > 0; j >>= 1) {
      const uint32_t o = __shfl_xor_sync(0xffffffffu, k, j);
      k = ((lane & size) == 0) == ((lane & j) == 0) ? max(k, o) : min(k, o);
    }
  }
  return k;
}

// Elements [v0, v1) of a row whose key is k, the first `want` of them in the order of their indexes, to the
// block's words.
template <bool kBF16, int NT>
__device__ __noinline__ void first_equal(const RowView<kBF16>& x, int v0, int v1, uint32_t k, uint32_t want, Few<true, NT>& sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int base = v0; base < v1 && want > 0; base += NT) {
    const int v = base + static_cast<int>(threadIdx.x);
    const bool is = v < v1 && fkey(clean(x.at(v))) == k;
    const unsigned who = __ballot_sync(0xffffffffu, is);
    __syncthreads();
    if (lane == 0) sm.ties[warp] = __popc(who);
    __syncthreads();
    uint32_t before = 0, all = 0;
    for (int i = 0; i < NT / 32; ++i) {
      before += i < warp ? sm.ties[i] : 0u;
      all += sm.ties[i];
    }
    before += __popc(who & ((1u << lane) - 1u));
    if (is && before < want) sm.words[atomicAdd(&sm.n_words, 1u)] = word_of(k, v);
    want -= min(want, all);
  }
}

// The first n of the block's part of a row, in any order and with others perhaps, to words: vectors [g0, g1),
// of which the thread's largest element is `most`, in its round that starts at vector `at`, and the largest of its
// other rounds `next`; and `loose`, its element outside the vectors (index loose_v; -inf: none).  [v0, v1) is all
// of the part.  False where there is no room for them.  Ends with a barrier.
template <bool kBF16, int NT>
__device__ __forceinline__ bool gather_words(const RowView<kBF16>& x, int g0, int g1, int v0, int v1, float most, int at, float next,
                                             float loose, int loose_v, int n, Few<true, NT>& sm) {
  constexpr int G = kBF16 ? 8 : 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kPer = kFew / (NT / 32), kU = kLoads<NT>;
  const uint32_t mine = fkey(most + 0.0f);
  {
    uint32_t k = mine;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint32_t top = __reduce_max_sync(0xffffffffu, k);
      if (lane == 0) sm.tops[kPer * warp + i] = top;
      if (lane == __ffs(__ballot_sync(0xffffffffu, k == top)) - 1) k = 0u;
    }
  }
  if (threadIdx.x == 0) sm.n_words = sm.n_who[0] = sm.n_who[1] = 0u;
  __syncthreads();
  const uint32_t bound = __shfl_sync(0xffffffffu, sort_warp(sm.tops[lane]), n - 1);
  auto collect = [&](uint32_t from) {
    auto take = [&](const uint4& v, int g) {
      if (fkey(no_nan(vec_max<kBF16>(v)) + 0.0f) < from) return;
#pragma unroll
      for (int e = 0; e < G; ++e) {
        const uint32_t k = fkey(clean(elem<kBF16>(v, e)));
        if (k < from) continue;
        const uint32_t pos = atomicAdd(&sm.n_words, 1u);
        if (pos < static_cast<uint32_t>(kWords)) sm.words[pos] = word_of(k, x.head + g * G + e);
      }
    };
    if (mine >= from) {
      const int which = fkey(next + 0.0f) >= from ? 1 : 0;
      sm.who[which][atomicAdd(&sm.n_who[which], 1u)] = static_cast<uint16_t>(threadIdx.x);
      sm.at[threadIdx.x] = at;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < static_cast<int>(sm.n_who[0]) * kU; i += NT) {
      const int who = sm.who[0][i / kU], u = i % kU;
      take(sm.kept[u][who], sm.at[who] + u * NT + who);
    }
    const int rounds = (g1 - g0 + NT - 1) / NT, items = static_cast<int>(sm.n_who[1]) * rounds;
    const float each = 1.0f / static_cast<float>(rounds);  // (i + 1/2 over rounds: whole parts are right below 2^22)
    for (int i = threadIdx.x; i < items; i += NT) {
      const int h = static_cast<int>((static_cast<float>(i) + 0.5f) * each), g = g0 + (i - h * rounds) * NT + sm.who[1][h];
      if (g < g1) take(x.vec[g], g);
    }
    const uint32_t k = fkey(clean(loose));
    if (k >= from) {
      const uint32_t pos = atomicAdd(&sm.n_words, 1u);
      if (pos < static_cast<uint32_t>(kWords)) sm.words[pos] = word_of(k, loose_v);
    }
    __syncthreads();
  };
  // (of a bound of -inf: everything above; what else is needed is found below.)  Where many elements equal the
  // bound, only larger ones.
  uint32_t tie = kKeyNegInf, from = max(bound, kKeyNegInf + 1u);
#pragma unroll 1
  for (int again = 0; again < 2; ++again) {
    collect(from);
    if (sm.n_words <= static_cast<uint32_t>(kWords) || bound == kKeyNegInf || again) break;
    __syncthreads();
    if (threadIdx.x == 0) sm.n_words = sm.n_who[0] = sm.n_who[1] = 0u;
    __syncthreads();
    tie = bound;
    from = bound + 1u;
  }
  const uint32_t have = sm.n_words;
  if (have > static_cast<uint32_t>(kWords)) return false;
  if (have < static_cast<uint32_t>(n)) first_equal<kBF16, NT>(x, v0, v1, tie, static_cast<uint32_t>(n) - have, sm);
  __syncthreads();
  return true;
}

// The first n of count words in their order, to out (distinct; by the whole block).
template <int NT>
__device__ __forceinline__ void rank_words(const unsigned long long* words, int count, int n, unsigned long long* out) {
  for (int i = threadIdx.x; i < count; i += NT) {
    const unsigned long long w = words[i];
    int r = 0;
#pragma unroll 4
    for (int j = 0; j < count; ++j) r += words[j] > w ? 1 : 0;
    if (r < n) out[r] = w;
  }
}

template <bool kBF16, bool kList, int NT>
__global__ void __launch_bounds__(NT, NT == 512 ? 2 : 5 * 256 / NT) score_kernel(const Args A) {
  constexpr int G = kBF16 ? 8 : 4, NW = NT / 32, kU = kLoads<NT>;
  __shared__ Part part[kWidest<NT> * NW];  // of the cluster's warps (rank 0's are used)
  __shared__ Few<kList, NT> sm;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  cg::cluster_group cl = cg::this_cluster();
  const int CS = static_cast<int>(cl.num_blocks());
  const int rank = static_cast<int>(cl.block_rank());
  const int64_t row = blockIdx.x / CS;
  const int n = A.n;
  // every CTA of the cluster runs before any writes into another's shared memory
  if (CS > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  const RowView<kBF16> x(A.x, row * A.ld, A.V);
  const int g0 = static_cast<int>(static_cast<int64_t>(x.nv) * rank / CS);
  const int g1 = static_cast<int>(static_cast<int64_t>(x.nv) * (rank + 1) / CS);
  // The first round is on its way to the second-level cache before the token says that the row counts; a row of
  // padding costs its first round (at most 20 KB a block), which is fetched but not looked at.  Graph replays with and
  // without, us: rows of fp32 without alternatives, 4096 x 32000 79.1 and 84.1, 1024 x 128256 82.8 and 84.2, 333 x 50001
  // 13.4 and 14.9; of bf16, 4096 x 151936 187.0 and 189.3, 2048 x 128256 87.8 and 89.2, 333 x 50001 13.1 and 13.6; with
  // five alternatives 2048 x 128256 bf16 105.7 and 109.3, 2048 x 32000 fp32 54.0 and 58.8; 8192 x 5000 is the same to 1%.
  // With a quarter of padding: 4096 x 151936 bf16 145.1 and 147.3 (as calls, other inputs each, 151.9 and 150.5), 4096 x
  // 32000 fp32 65.7 and 64.8; with half 47.6 and 44.8, and 2048 x 128256 bf16 with five alternatives 66.0 and 67.5.
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int g = g0 + u * NT + static_cast<int>(threadIdx.x);
    if (g < g1) asm volatile("prefetch.global.L2 [%0];" ::"l"(x.vec + g));
  }
  const int64_t t = A.tokens[row];
  const float tau = row_tau(A.taus, A.tau, row);
  if (t < 0 || t >= A.V || (A.weight && A.weight[row] == 0.0f)) {  // an empty row
    if (CS > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (rank == 0) put_empty(A, row, NT);
    return;
  }
  const float token = no_nan(x.at(static_cast<int>(t)));
  const float c = kLog2e / tau;

  Moments<kBF16> sum;
  float top = -INFINITY;  // the warp's largest so far; the sums' reference (0 before there is one)
  const f32x2 c2 = pack2(c, c);
  f32x2 nref2 = 0ull;
  float above = 0.0f;
  // The reference rises to `to`; the element that held it joins the sums.
  auto raise = [&](float to) {
    if (top > -INFINITY) {
      const float delta = fminf((to - top) * c, -kFloor);
      sum.shift(delta);
      if (lane == 0) {
        const float e = ex2(-delta);
        sum.s[0] = add2(sum.s[0], pack2(e, 0.0f));
        sum.w[0] = add2(sum.w[0], pack2(-delta * e, 0.0f));
      }
    }
    top = to;
    nref2 = pack2(-to, -to);
  };
  // the elements outside the vectors, by one warp: the head with rank 0, the tail with the last rank
  const bool in = warp == 0 && lane < x.loose() && ((x.loose_at(lane) < x.head) ? rank == 0 : rank == CS - 1);
  float loose = in ? x.at(x.loose_at(lane)) : -INFINITY;
  const float outside = loose;

  float thread_top = -INFINITY, thread_next = -INFINITY;  // of this thread's rounds, and of all but that one
  int top_at = g0;
  // a round of loads; only the last one has to look where the CTA's part ends
  auto round = [&](int base, auto full) {
    constexpr bool kFull = decltype(full)::value;
    uint4 w[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int g = base + u * NT + static_cast<int>(threadIdx.x);
      w[u] = kFull || g < g1 ? ld_stream(x.vec + g) : neg_inf_vec<kBF16>();
    }
    float m[kU], most = -INFINITY;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      m[u] = vec_max<kBF16>(w[u]);
      most = fmaxf(most, m[u]);
      if (m[u] > token) above += count_above<kBF16>(w[u], token);
    }
    if constexpr (kList) {
      thread_next = fmaxf(thread_next, fminf(thread_top, most));
      if (most > thread_top) {
        thread_top = most;
        top_at = base;
#pragma unroll
        for (int u = 0; u < kU; ++u) sm.kept[u][threadIdx.x] = w[u];
      }
    }
    if (__any_sync(0xffffffffu, most > top)) {
      const float to = warp_top(most);
      raise(to);
      const unsigned who = __ballot_sync(0xffffffffu, most == to);
      if (lane == __ffs(who) - 1) {
        bool done = false;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          if (done || m[u] != to) continue;
          strike<kBF16>(w[u], to);
          done = true;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) sum.add(w[u], nref2, c2);
  };
  int base = g0;
#pragma unroll 1
  for (; base + NT * kU <= g1; base += NT * kU) round(base, std::true_type{});
  if (base < g1) round(base, std::false_type{});
  float extra = 0.0f, extra_w = 0.0f;
  if (warp == 0) {
    if (loose > token) above += 1.0f;
    if (__any_sync(0xffffffffu, loose > top)) {
      const float to = warp_top(loose);
      raise(to);
      const unsigned who = __ballot_sync(0xffffffffu, loose == to);
      if (lane == __ffs(who) - 1) loose = -INFINITY;
    }
    const float z = exponent(loose, top == -INFINITY ? 0.0f : top, c);
    extra = ex2(z);
    extra_w = extra * z;
  }
  const float s = warp_sum(extra + sum.sum()), moment = warp_sum(extra_w + sum.moment());
  above = warp_sum(above);
  Part* to = CS > 1 ? cl.map_shared_rank(&part[0], 0) : part;
  if (CS > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (lane == 0) to[rank * NW + warp] = Part{top, s, moment, above};
  if constexpr (kList) {
    const int v0 = rank == 0 ? 0 : x.head + g0 * G, v1 = rank == CS - 1 ? A.V : x.head + g1 * G;
    const bool whole = gather_words<kBF16, NT>(x, g0, g1, v0, v1, thread_top, top_at, thread_next, outside, x.loose_at(lane), n, sm);
    unsigned long long* best = CS > 1 ? cl.map_shared_rank(&sm.lists[0][0], 0) + rank * kFew : sm.best;
    if (whole) rank_words<NT>(sm.words, static_cast<int>(sm.n_words), n, best);
    if (threadIdx.x == 0)
      *(CS > 1 ? cl.map_shared_rank(&sm.sizes[0], 0) + rank : &sm.sizes[0]) = whole ? min(sm.n_words, static_cast<uint32_t>(n)) : ~0u;
  }
  if (CS > 1) {
    cl.sync();
    if (rank != 0) return;
  } else {
    __syncthreads();
  }
  if constexpr (kList) {
    bool whole = true;
    for (int i = 0; i < CS; ++i) whole = whole && sm.sizes[i] != ~0u;
    if (!whole) {
      exact_select<kBF16, NT>(x, n, 0u, c, sm);  // (its sum is not needed)
      __syncthreads();
      rank_words<NT>(sm.words, n, n, sm.best);
    } else if (CS > 1) {
      // the CTAs' lists one behind the other
      int at = 0;
      for (int i = 0; i < CS; ++i) {
        const int size = static_cast<int>(sm.sizes[i]);
        if (static_cast<int>(threadIdx.x) < size) sm.words[at + threadIdx.x] = sm.lists[i][threadIdx.x];
        at += size;
      }
      __syncthreads();
      rank_words<NT>(sm.words, at, n, sm.best);
    }
    __syncthreads();
  }
  if (warp != 0) return;
  // the parts' sums against the row's largest logit; the first part that holds it keeps it out
  static_assert(kWidest<NT> * NW <= 64);
  const Part none{-INFINITY, 0.0f, 0.0f, 0.0f};
  const Part p0 = lane < NW * CS ? part[lane] : none, p1 = lane + 32 < NW * CS ? part[lane + 32] : none;
  const float m = warp_top(fmaxf(p0.m, p1.m));
  const unsigned w0 = __ballot_sync(0xffffffffu, p0.m == m), w1 = __ballot_sync(0xffffffffu, p1.m == m);
  const int owner = w0 ? __ffs(w0) - 1 : 32 + __ffs(w1) - 1;
  float s0, s1, m0, m1;
  part_to_row(p0, lane == owner, m, c, s0, m0);
  part_to_row(p1, lane + 32 == owner, m, c, s1, m1);
  const Row r(m, warp_sum(s0 + s1), warp_sum(m0 + m1));
  above = warp_sum(p0.above + p1.above);
  if (lane == 0) put_row(A, row, r, token, tau, above);
  if constexpr (kList) {
    if (lane < n) {
      A.ids[row * n + lane] = word_index(sm.best[lane]);
      A.logprobs[row * n + lane] = r.logprob(word_value(sm.best[lane]), tau);
    }
  }
}

// ------------------------------------------------------------------------------------------
// The gradient
// ------------------------------------------------------------------------------------------
struct Grad {
  Args a;             // max, eps, q are read
  const float* g;     // the gradients of the log-probability and the entropy, or nullptr: 0
  const float* h;
  void* out;
  int64_t ld_out;
  // the policy loss (kPolicy): a.max, a.eps, a.q lie in loss, a.logprob, a.entropy, which are written last
  const float *old, *advantage, *ref;  // ref: or nullptr
  float lo, hi, kl, ent;
  float* loss;
};

// exp(u) - u - 1 for all u: near 0 by its series, u^2/2! + u^3/3! + ...
__device__ __forceinline__ float expm1_minus(float u) {
  if (!(fabsf(u) < 0.5f)) return u == INFINITY ? INFINITY : expm1f(u) - u;
  float t = 1.0f;  // 1 + u/3 (1 + u/4 (... (1 + u/11))): the next factor is below 2^-28 of the sum
#pragma unroll
  for (int i = 11; i >= 3; --i) t = fmaf(t * u, 1.0f / static_cast<float>(i), 1.0f);
  return 0.5f * u * u * t;
}

// What a row's loss needs beside its logits.
struct PolicyRow {
  float w, A, old, ref;
  __device__ __forceinline__ PolicyRow(const Grad& P, int64_t row) {
    w = P.a.weight ? P.a.weight[row] : 1.0f;
    A = P.advantage[row];
    old = P.old[row];
    ref = P.kl != 0.0f ? P.ref[row] : 0.0f;
  }
};
// A row's loss and the gradients of its log-probability and entropy.
struct PolicyTerm {
  float loss, g, h;
  __device__ __forceinline__ PolicyTerm(const Grad& P, const PolicyRow& in, float logprob, float entropy) {
    const float A = in.A, w = in.w, r = expf(logprob - in.old);
    const float kept = fminf(fmaxf(r, 1.0f - P.lo), 1.0f + P.hi);
    const bool clipped = A >= 0.0f ? r > 1.0f + P.hi : A < 0.0f && r < 1.0f - P.lo;  // (NaN: not)
    float v = 0.0f, d = 0.0f;
    if (A != 0.0f || isnan(r)) {  // (an infinite ratio times an advantage of 0 is 0; a NaN in either stays)
      v = -(clipped ? kept : r) * A;
      d = clipped ? 0.0f : -A * r;
    }
    if (P.kl != 0.0f) {
      const float u = in.ref - logprob;
      v += P.kl * expm1_minus(u);
      d -= P.kl * expm1f(u);
    }
    if (P.ent != 0.0f) v -= P.ent * entropy;
    if (isnan(logprob)) v = NAN;
    loss = w * v;
    g = w * d;
    h = -w * P.ent;
  }
};

// At temperatures below 2^-60 g / tau and h / tau may leave fp32 while the gradient does not: between equal logits, of
// which there are up to 2^20, it is that part of them, and beside a certain token 0.  So a slope is held 2^-20 down
// there, for g and h below 2^22 at least, and its elements are taken one at a time and brought up by whoever writes them.
// (At every temperature it would cost the smallest gradients their last bits.)
__device__ __forceinline__ bool is_tiny(float c) { return c > kLog2e * 0x1p60f; }
__device__ __forceinline__ float slope_up(float c) { return is_tiny(c) ? 0x1p20f : 1.0f; }

// A row's gradient over slope_up: e_v (A + B z_v) with e_v = 2^z_v, z_v = (x_v - m) c; the token's apart.
struct Slope {
  float a, b, token;
  __device__ __forceinline__ Slope(float a_, float b_, float token_) : a(a_), b(b_), token(token_) {}
  __device__ __forceinline__ Slope(const Row& r, float x_token, float tau, float c, float g, float h) {
    const float inv = 1.0f / (1.0f + r.eps);
    const float by = tau * slope_up(c), gt = g / by, ht = h / by;
    a = r.ok ? -(gt + ht * r.q) * inv : NAN;
    b = h == 0.0f ? 0.0f : -ht * kLn2 * inv;
    // the token's: 1 - p without the difference of two ones where it is the largest
    const float z = exponent(x_token, r.m, c), e = ex2(z);
    const float rest = z == 0.0f ? r.eps * inv : 1.0f - e * inv;
    token = r.ok ? gt * rest + (h == 0.0f ? 0.0f : -ht * (e * inv) * (r.q + kLn2 * z)) : NAN;
  }
  __device__ __forceinline__ float at(float x, float m, float c) const {
    const float z = exponent(x, m, c), e = ex2(z);
    return e == 0.0f ? 0.0f : fmaf(b, z, a) * e;
  }
  // Whether a + b z is finite for every z from kFloor on; else only at() is.
  __device__ __forceinline__ bool tame() const { return fabsf(a) < 0x1p110f && fabsf(b) < 0x1p110f; }
};
template <bool kBF16>
__device__ __forceinline__ void put_elem(void* base, int64_t v, float d) {
  if (kBF16) static_cast<__nv_bfloat16*>(base)[v] = __float2bfloat16_rn(d);
  else static_cast<float*>(base)[v] = d;
}
// Zeros to a CTA's part of a row of the gradient.
template <bool kBF16>
__device__ __forceinline__ void zero_part(const RowView<kBF16>& o, int rank, int CS) {
  const int o0 = static_cast<int>(static_cast<int64_t>(o.nv) * rank / CS);
  const int o1 = static_cast<int>(static_cast<int64_t>(o.nv) * (rank + 1) / CS);
  uint4* ov = const_cast<uint4*>(o.vec);
  for (int i = o0 + static_cast<int>(threadIdx.x); i < o1; i += kNT) __stcs(ov + i, make_uint4(0u, 0u, 0u, 0u));
  if (rank == 0 && static_cast<int>(threadIdx.x) < o.loose())
    put_elem<kBF16>(const_cast<unsigned char*>(o.base), o.loose_at(threadIdx.x), 0.0f);
}
// The gradient of a vector's elements.  Without b one multiply-add an exponent does, as nothing cancels:
// x c - rc with rc the rounded product of m and c, put right in a.
template <bool kBF16>
struct SlopeVec {
  f32x2 c2, n2, a2, b2;
  bool flat, usable;  // b is 0; the vectors' way does for this row
  __device__ __forceinline__ SlopeVec(const Slope& s, float m, float c) {
    const float rc = m * c;
    flat = s.b == 0.0f && fabsf(rc) <= kFastRef;
    const float a = flat ? s.a * ex2(-fmaf(m, c, -rc)) : s.a, n = flat ? -rc : -m;
    c2 = pack2(c, c);
    n2 = pack2(n, n);
    a2 = pack2(a, a);
    b2 = pack2(s.b, s.b);
    usable = s.tame() && !is_tiny(c);
  }
  static __device__ __forceinline__ void put(uint32_t* out, int i, float p, float q) {
    if (kBF16) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(p, q);  // the gradient's one rounding
      out[i] = reinterpret_cast<const uint32_t&>(h);
    } else {
      out[2 * i] = __float_as_uint(p);
      out[2 * i + 1] = __float_as_uint(q);
    }
  }
  template <bool kFlat, bool kFree = false>
  __device__ __forceinline__ uint4 of(const uint4& v) const {
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < (kBF16 ? 4 : 2); ++i) {
      const f32x2 x = pair_of<kBF16>(v, i);
      float p, q;
      if (kFlat) {
        unpack2(fma2(x, c2, n2), p, q);
        unpack2(mul2(pack2(ex2(p), ex2(q)), a2), p, q);
      } else {
        unpack2(mul2(add2(x, n2), c2), p, q);
        if (!kFree) {
          p = max_nan(p, kFloor);
          q = max_nan(q, kFloor);
        }
        unpack2(mul2(pack2(ex2(p), ex2(q)), fma2(b2, pack2(p, q), a2)), p, q);
      }
      put(out, i, p, q);
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
  }
};

// 2048 rows of 128256 bf16, a quarter of them empty: 134 us (138 at the copy rate) in up to eight CTAs a row, with
// four loads in flight and six CTAs an SM; six and four 147, three and eight 138, two and eight 136; six and four
// with one CTA a row 141.  333 rows of 50001 fp32: 21.9 us, and 24.0, 21.9, 22.7, 23.3.
template <bool kBF16, bool kPolicy>
__global__ void __launch_bounds__(kNT, 6) slope_kernel(const Grad P) {
  constexpr int kU = 4;  // loads in flight
  constexpr int G = kBF16 ? 8 : 4;
  const Args& A = P.a;
  cg::cluster_group cl = cg::this_cluster();
  const int CS = static_cast<int>(cl.num_blocks());
  const int rank = static_cast<int>(cl.block_rank());
  const int64_t row = blockIdx.x / CS;
  const RowView<kBF16> x(A.x, row * A.ld, A.V), o(P.out, row * P.ld_out, A.V);
  unsigned char* const obase = const_cast<unsigned char*>(o.base);
  const int64_t t = A.tokens[row];
  const float tau = row_tau(A.taus, A.tau, row), c = kLog2e / tau;
  float g = 0.0f, h = 0.0f;
  bool live = t >= 0 && t < A.V;
  if constexpr (kPolicy) {
    live = live && !(A.weight && A.weight[row] == 0.0f);
  } else {
    if (P.g) g = P.g[row];
    if (P.h) h = P.h[row];
    live = live && (g != 0.0f || h != 0.0f);
  }
  if (!live) {  // zeros; the row is not looked at (the same in every CTA of the row)
    zero_part<kBF16>(o, rank, CS);
    if (kPolicy && rank == 0 && threadIdx.x == 0) P.loss[row] = A.logprob[row] = A.entropy[row] = 0.0f;
    return;
  }
  const Row r(A.max, A.eps, A.q, row);
  const float x_token = x.at(static_cast<int>(t));
  if constexpr (kPolicy) {
    const float logprob = r.logprob(x_token, tau), entropy = r.entropy();
    const PolicyTerm term(P, PolicyRow(P, row), logprob, entropy);
    g = term.g;
    h = term.h;
    if (CS > 1) cl.sync(); else __syncthreads();  // every thread of the row has read its statistics
    if (rank == 0 && threadIdx.x == 0) {
      P.loss[row] = term.loss;
      A.logprob[row] = logprob;
      A.entropy[row] = entropy;
    }
  }
  const Slope slope(r, x_token, tau, c, g, h);
  const int g0 = static_cast<int>(static_cast<int64_t>(x.nv) * rank / CS);
  const int g1 = static_cast<int>(static_cast<int64_t>(x.nv) * (rank + 1) / CS);
  const int at = static_cast<int>(t) - x.head;  // the token's vector, if it is in one
  const int tv = at >= 0 && at < x.nv * G ? at / G : -1;
  const SlopeVec<kBF16> vec(slope, r.m, c);
  if (o.head == x.head && vec.usable) {
    uint4* ov = const_cast<uint4*>(o.vec);
    auto round = [&](int base, auto flat, auto full) {
      constexpr bool kFull = decltype(full)::value;
      uint4 v[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int i = base + u * kNT + static_cast<int>(threadIdx.x);
        v[u] = kFull || i < g1 ? ld_stream(x.vec + i) : neg_inf_vec<kBF16>();
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int i = base + u * kNT + static_cast<int>(threadIdx.x);
        if (kFull || i < g1) __stcs(ov + i, vec.template of<decltype(flat)::value>(v[u]));
        if (i == tv && i < g1) put_elem<kBF16>(obase, t, slope.token);  // by the thread that wrote the vector, behind it
      }
    };
    auto pass = [&](auto flat) {
      int base = g0;
#pragma unroll 1
      for (; base + kNT * kU <= g1; base += kNT * kU) round(base, flat, std::true_type{});
      if (base < g1) round(base, flat, std::false_type{});
    };
    if (vec.flat) pass(std::true_type{});
    else pass(std::false_type{});
    if (static_cast<int>(threadIdx.x) < x.loose()) {
      const int v = x.loose_at(threadIdx.x);
      if ((v < x.head) ? rank == 0 : rank == CS - 1) put_elem<kBF16>(obase, v, slope_up(c) * (v == t ? slope.token : slope.at(x.at(v), r.m, c)));
    }
  } else {
    // the two rows do not share their 16-byte boundaries, or the numbers are extreme: one element at a time
    const int v0 = rank == 0 ? 0 : x.head + g0 * G, v1 = rank == CS - 1 ? A.V : x.head + g1 * G;
    for (int v = v0 + static_cast<int>(threadIdx.x); v < v1; v += kNT)
      put_elem<kBF16>(obase, v, slope_up(c) * (v == t ? slope.token : slope.at(x.at(v), r.m, c)));
  }
}

// ------------------------------------------------------------------------------------------
// The policy loss with the row in shared memory
// ------------------------------------------------------------------------------------------
//
// The row is read once, by a bulk copy into the shared memory of each of a cluster's CTAs, summed
// there against the CTA's largest logit, turned into the gradient in place and copied out.
// Bytes of a row per CTA, where the cluster allows: five CTAs an SM (48 registers).  4096 rows of 151936 bf16
// with a quarter empty take 365 us (326 at the copy rate), 2048 of 128256 180 (157); with 52 KB and four CTAs 371
// and 184, with 62 KB and three 427 and 224 at the time.  Loops unrolled more than twice cost 2% (instructions
// are fetched anew by every block), parts copied in and out in two slices 1%, in four 5%.
constexpr int kChunkBytes = 43 * 1024;

template <bool kBF16>
__global__ void __launch_bounds__(kNT, 5) policy_kernel(const Grad P, const int share) {
  constexpr int G = kBF16 ? 8 : 4;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float sums[kMaxCS * kNW][2];  // S and W of the cluster's warps
  __shared__ float tops[kMaxCS];           // the CTAs' largest logits
  __shared__ uint32_t keys[kNW];
  __shared__ float factors[4];             // m, a, b and the token's gradient
  __shared__ __align__(8) unsigned long long landed, gathered;  // the barriers of the copy and of sums and tops
  const Args& A = P.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  cg::cluster_group cl = cg::this_cluster();
  const int CS = static_cast<int>(cl.num_blocks());
  const int rank = static_cast<int>(cl.block_rank());
  uint32_t cluster;
  asm("mov.u32 %0, %%clusterid.x;" : "=r"(cluster));
  const int64_t row = cluster;
  if (threadIdx.x == 0) {
    copy_barrier_init(&landed);
    copy_barrier_init(&gathered);
    expect_bytes(&gathered, static_cast<uint32_t>(CS * (2 * kNW + 1) * sizeof(float)));
  }
  __syncwarp();
  // every CTA of the cluster runs, and has set up its barriers, before any writes into another's
  // shared memory (the barriers' own fence is behind their setting up)
  if (CS > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const RowView<kBF16> x(A.x, row * A.ld, A.V), o(P.out, row * P.ld_out, A.V);
  unsigned char* const obase = const_cast<unsigned char*>(o.base);
  const int g0 = min(rank * share, x.nv), g1 = rank == CS - 1 ? x.nv : min(g0 + share, x.nv);
  uint4* const mine = reinterpret_cast<uint4*>(smem) + threadIdx.x;  // the thread's vectors: mine[i kNT], i < count
  const int first = g0 + static_cast<int>(threadIdx.x), count = first < g1 ? (g1 - first - 1) / kNT + 1 : 0;
  const int64_t t = A.tokens[row];
  if (t < 0 || t >= A.V || (A.weight && A.weight[row] == 0.0f)) {  // an empty row: zeros (the same in every CTA of the row)
    if (CS > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    zero_part<kBF16>(o, rank, CS);
    if (rank == 0 && threadIdx.x == 0) P.loss[row] = A.logprob[row] = A.entropy[row] = 0.0f;
    return;
  }
  if (threadIdx.x == 0 && g1 > g0) copy_in(smem, x.vec + g0, static_cast<uint32_t>(g1 - g0) * 16u, &landed);
  const float c = kLog2e / row_tau(A.taus, A.tau, row);
  const PolicyRow inputs(P, row);
  const float x_token = x.at(static_cast<int>(t));
  // the elements outside the vectors: the head with rank 0, the tail with the last rank
  const bool has_loose = static_cast<int>(threadIdx.x) < x.loose() &&
                         ((x.loose_at(threadIdx.x) < x.head) ? rank == 0 : rank == CS - 1);
  const int loose_v = has_loose ? x.loose_at(threadIdx.x) : 0;
  float loose_x = has_loose ? x.at(loose_v) : -INFINITY;
  __syncthreads();  // the barriers are set up
  const bool late = __any_sync(0xffffffffu, g1 > g0 && !copy_landed(&landed));  // the wait ran out

  // ---- the CTA's largest logit, and the thread that holds it ---------------------------------------
  uint4 best = neg_inf_vec<kBF16>(), least = make_uint4(0u, 0u, 0u, 0u);  // (no smallest above 0 is needed)
#pragma unroll 2
  for (int i = 0; i < count; ++i) {
    const uint4 v = mine[i * kNT];
    best = vec_extreme<kBF16>(best, v);
    least = vec_extreme<kBF16, true>(least, v);
  }
  const float bottom = vec_min<kBF16>(least);
  const float own = vec_max<kBF16>(best), most = fmaxf(no_nan(loose_x), no_nan(own));
  const uint32_t key = fkey(most + 0.0f), warp_key = __reduce_max_sync(0xffffffffu, key);
  if (lane == 0) keys[warp] = warp_key;
  __syncthreads();
  const uint32_t other = keys[lane & (kNW - 1)], top_key = __reduce_max_sync(0xffffffffu, other);
  const float top = kfloat(top_key);
  const bool here = warp == __ffs(__ballot_sync(0xffffffffu, other == top_key)) - 1;
  const bool holds = here && lane == __ffs(__ballot_sync(0xffffffffu, key == top_key)) - 1;

  // ---- the sums of everything else -----------------------------------------------------------------
  const float ref = top > -INFINITY ? top : 0.0f;
  {
    Moments<kBF16> sum;
    const f32x2 nref2 = pack2(-ref, -ref), c2 = pack2(c, c);
    bool skip = holds;  // the element that stays out is still to come
    if (skip && loose_x == top) {
      loose_x = -INFINITY;
      skip = false;
    }
    if (!here && __all_sync(0xffffffffu, (bottom - ref) * c >= kFloor)) {
#pragma unroll 2
      for (int i = 0; i < count; ++i) sum.template add<true>(mine[i * kNT], nref2, c2);
    } else {
#pragma unroll 2
      for (int i = 0; i < count; ++i) {
        uint4 v = mine[i * kNT];
        if (skip && vec_max<kBF16>(v) == top) {
          strike<kBF16>(v, top);
          skip = false;
        }
        sum.add(v, nref2, c2);
      }
    }
    const float z = exponent(loose_x, ref, c), e = ex2(z);
    float s = warp_sum(e + sum.sum());
    const float m1 = warp_sum(e * z + sum.moment());
    if (late) s = NAN;  // a part that did not arrive leaves its row without a result
    if (CS > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // (of the arrival at the top)
    if (lane < CS) {
      send_float(&sums[rank * kNW + warp][0], s, &gathered, lane);
      send_float(&sums[rank * kNW + warp][1], m1, &gathered, lane);
      if (warp == 0) send_float(&tops[rank], top, &gathered, lane);
    }
  }

  // ---- the row's statistics, its loss and the gradient's factors, by one warp ------------------------
  if (warp == 0) {
    const bool lost = !copy_landed(&gathered);
    float m = lane < CS ? tops[lane] : -INFINITY;
    m = warp_top(m);
    const int owner = __ffs(__ballot_sync(0xffffffffu, lane < CS && tops[lane & (kMaxCS - 1)] == m)) - 1;
    float s = 0.0f, m1 = 0.0f;
    for (int i = lane; i < kNW * CS; i += 32) {
      const int cta = i / kNW;
      float a, b;  // (a CTA's largest element enters with its first warp)
      part_to_row(Part{tops[cta], sums[i][0], sums[i][1], 0.0f}, i % kNW != 0 || cta == owner, m, c, a, b);
      s += a;
      m1 += b;
    }
    s = warp_sum(s);
    m1 = warp_sum(m1);
    const Row r(m, lost ? NAN : s, m1);
    const float tau = row_tau(A.taus, A.tau, row);
    const float logprob = r.logprob(x_token, tau), entropy = r.entropy();
    const PolicyTerm term(P, inputs, logprob, entropy);
    const Slope slope(r, x_token, tau, c, term.g, term.h);
    if (lane == 0) {
      factors[0] = r.m;
      factors[1] = slope.a;
      factors[2] = slope.b;
      factors[3] = slope.token;
      if (rank == 0) {
        P.loss[row] = term.loss;
        A.logprob[row] = logprob;
        A.entropy[row] = entropy;
      }
    }
  }
  __syncthreads();

  // ---- the gradient: in place in shared memory, and out with one copy --------------------------------
  const float m = factors[0];
  const Slope slope(factors[1], factors[2], factors[3]);
  const int v0 = x.head + g0 * G, v1 = x.head + g1 * G;  // this CTA's vectors
  const bool inside = t >= v0 && t < v1;
  const SlopeVec<kBF16> vec(slope, m, c);
  if (o.head == x.head && vec.usable) {
    if (vec.flat) {
#pragma unroll 2
      for (int i = 0; i < count; ++i) mine[i * kNT] = vec.template of<true>(mine[i * kNT]);
    } else if (__all_sync(0xffffffffu, (bottom - m) * c >= kFloor)) {
#pragma unroll 2
      for (int i = 0; i < count; ++i) mine[i * kNT] = vec.template of<false, true>(mine[i * kNT]);
    } else {
      for (int i = 0; i < count; ++i) mine[i * kNT] = vec.template of<false>(mine[i * kNT]);
    }
    if (inside && (static_cast<int>(t) - v0) / G % kNT == static_cast<int>(threadIdx.x))
      put_elem<kBF16>(smem, t - v0, slope.token);  // behind the vector, by the same thread
    publish_to_copies();
    __syncthreads();
    if (threadIdx.x == 0 && g1 > g0) copy_out(const_cast<uint4*>(o.vec) + g0, smem, static_cast<uint32_t>(g1 - g0) * 16u);
  } else {
    // the two rows do not share their 16-byte boundaries, or the numbers are extreme: one element at a time (unrolled,
    // its instructions cost every block 0.4%)
#pragma unroll 1
    for (int v = v0 + static_cast<int>(threadIdx.x); v < v1; v += kNT) {
      const float y = kBF16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(smem)[v - v0]) : reinterpret_cast<const float*>(smem)[v - v0];
      put_elem<kBF16>(obase, v, slope_up(c) * (v == t ? slope.token : slope.at(y, m, c)));
    }
  }
  if (has_loose) put_elem<kBF16>(obase, loose_v, slope_up(c) * (loose_v == t ? slope.token : slope.at(x.at(loose_v), m, c)));
  if (late) copy_landed(&landed);  // one more wait before the block leaves
}

// ------------------------------------------------------------------------------------------
// Host side
// ------------------------------------------------------------------------------------------
// Launches a kernel with a cluster of cs CTAs a row.
template <int NT = kNT, class... Params, class... Values>
static kps_status launch_clusters(void (*kernel)(Params...), int64_t N, int cs, size_t shared, cudaStream_t stream, const Values&... values) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(static_cast<unsigned>(N * cs));
  lc.blockDim = dim3(NT);
  lc.dynamicSmemBytes = shared;
  lc.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  if (cudaLaunchKernelEx(&lc, kernel, values...) == cudaSuccess) return KPS_OK;
  (void)cudaGetLastError();
  return KPS_ERR_CUDA;
}
// A streaming kernel: one CTA a row, or up to kMaxCS while there are no more than `fill` an SM (0: any number) and every thread keeps
// four vectors.  Five an SM for scoring without alternatives (256 rows of 151936 bf16: 21.6 us, 23.9 with two an SM;
// 333 of 50001 fp32 13.7 and 15.1), four with them (128 rows of 151936 bf16 19.2 and 19.8, 100 of 50001 fp32 12.3
// and 13.1).  The gradient's CTAs have nothing in common, so there it is as many as there can be.
template <class P>
static kps_status launch_rows(void (*kernel)(P), const Args& a, kps_dtype dt, int fill, int sms, const P& params, cudaStream_t stream) {
  int cs = 1;
  const int64_t round = static_cast<int64_t>(kNT) * 4 * (dt == KPS_BF16 ? 8 : 4);
  while (cs < kMaxCS && (fill == 0 || a.N * cs * 2 <= static_cast<int64_t>(fill) * sms) && a.V >= 2 * cs * round) cs *= 2;
  return launch_clusters(kernel, a.N, cs, 0, stream, params);
}
// Scoring.  Many short rows go to blocks of 128 threads, twice as many an SM, as a block spends some 3.5 us on
// its start and its end whatever its row is (8192 rows of 5000 bf16: 29.6 us; 27.8 and, with 256 threads, 44.5 when they
// were compared; with five alternatives 55 and 85; 2048 of 32000 bf16 30.9 and 33.7).  Rows above 64 KB are faster with
// 256 (2048 of 32000 fp32 with five alternatives 62 and 58.6, of 128256 bf16 125 and 109).  With alternatives, one or
// two long rows an SM go to blocks of 512 (256 of 151936 bf16, twenty alternatives: 26.5 us, 29.2 with 256 threads; 300
// of 128256 24.2 and 27.0; 200 of 50001 fp32 16.2 and 17.8): clusters of two of 256 take 28.7, 26.7 and 16.3.
constexpr int kShortBytes = 64 * 1024, kShortThreads = 128, kLongThreads = 512;
static kps_status launch_score(const Args& a, kps_dtype dt, cudaStream_t stream) {
  if (a.n > kFew) return launch_alternatives(a, dt, stream);
  const int sms = sm_count();
  if (!sms) return KPS_ERR_CUDA;
  const bool bf16 = dt == KPS_BF16, list = a.n > 0;
  if (a.N > 2 * sms && static_cast<int64_t>(a.V) * (bf16 ? 2 : 4) <= kShortBytes) {
    constexpr int NT = kShortThreads;
    auto* kernel = bf16 ? (list ? score_kernel<true, true, NT> : score_kernel<true, false, NT>)
                        : (list ? score_kernel<false, true, NT> : score_kernel<false, false, NT>);
    return launch_clusters<NT>(kernel, a.N, 1, 0, stream, a);
  }
  if (list && a.N > sms && a.N <= 2 * sms && static_cast<int64_t>(a.V) * (bf16 ? 2 : 4) > kShortBytes) {
    constexpr int NT = kLongThreads;
    return launch_clusters<NT>(bf16 ? score_kernel<true, true, NT> : score_kernel<false, true, NT>, a.N, 1, 0, stream, a);
  }
  auto* kernel = bf16 ? (list ? score_kernel<true, true, kNT> : score_kernel<true, false, kNT>)
                      : (list ? score_kernel<false, true, kNT> : score_kernel<false, false, kNT>);
  return launch_rows<Args>(kernel, a, dt, list ? 4 : 5, sms, a, stream);
}
template <bool kPolicy>
static kps_status launch_slope(const Grad& P, kps_dtype dt, cudaStream_t stream) {
  return launch_rows<Grad>(dt == KPS_BF16 ? slope_kernel<true, kPolicy> : slope_kernel<false, kPolicy>, P.a, dt, 0, 0, P, stream);
}

// The policy loss: with the row in shared memory where a cluster's holds it (up to 1.8 MB); longer rows
// are read twice, in two launches, and their statistics lie where the second leaves the results.
template <bool kBF16>
static kps_status launch_policy(const Grad& P, cudaStream_t stream) {
  constexpr int G = kBF16 ? 8 : 4;
  const int64_t bytes = static_cast<int64_t>(P.a.V) * (kBF16 ? 2 : 4);
  const int sms = sm_count();
  if (!sms) return KPS_ERR_CUDA;
  int cs = static_cast<int>((bytes + kChunkBytes - 1) / kChunkBytes);
  cs = cs < 1 ? 1 : cs > kMaxCS ? kMaxCS : cs;
  // few rows: wider clusters, while every thread keeps four vectors
  while (2 * cs <= kMaxCS && P.a.N * cs * 2 <= 2 * sms && P.a.V >= 2 * cs * kNT * 4 * G) cs *= 2;
  const int share = (P.a.V / G + cs - 1) / cs;
  const size_t total = static_cast<size_t>(share) * 16;
  if (total > kMaxDynamic) {
    const kps_dtype dt = kBF16 ? KPS_BF16 : KPS_F32;
    Grad two = P;
    two.a.max = P.loss;
    two.a.eps = P.a.logprob;
    two.a.q = P.a.entropy;
    Args a = two.a;
    a.logprob = a.entropy = nullptr;
    const kps_status st = launch_score(a, dt, stream);
    return st != KPS_OK ? st : launch_slope<true>(two, dt, stream);
  }
  static std::atomic<bool> done[kMaxDevices];
  if (!allow_shared(policy_kernel<kBF16>, done)) return KPS_ERR_CUDA;
  return launch_clusters(policy_kernel<kBF16>, P.a.N, cs, total, stream, P, share);
}

static bool misaligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

// The checks that every entry point shares; fills a.
static kps_status check(const void* logits, kps_dtype dt, int64_t N, int64_t V, int64_t ld, const int64_t* tokens,
                        float temperature, const float* temperatures, Args* a) {
  if (dt != KPS_F32 && dt != KPS_BF16) return KPS_ERR_INVALID_ARG;
  if (N < 0 || V < 1 || (N > 1 && ld < V)) return KPS_ERR_INVALID_ARG;
  if (!temperatures && (!(temperature > 0.0f) || std::isinf(temperature) || std::isinf(kLog2e / temperature))) return KPS_ERR_INVALID_ARG;
  if (V > kMaxV || N > INT32_MAX / kMaxCS) return KPS_ERR_UNSUPPORTED;
  if (N == 0) return KPS_OK;
  if (!logits || !tokens || misaligned(logits, dt == KPS_BF16 ? 2 : 4) || misaligned(tokens, 8) || misaligned(temperatures, 4))
    return KPS_ERR_INVALID_ARG;
  a->x = logits;
  a->N = N;
  a->ld = ld;
  a->V = static_cast<int>(V);
  a->tau = temperature;
  a->taus = temperatures;
  a->tokens = tokens;
  return KPS_OK;
}

}  // namespace score
}  // namespace kps

extern "C" {

kps_status kps_token_logprobs(const void* logits, kps_dtype dt, int64_t N, int64_t V, int64_t ld, const int64_t* tokens,
                              int64_t n, float temperature, const float* temperatures, float* out_logprob,
                              float* out_entropy, int32_t* out_rank, int32_t* out_ids, float* out_logprobs,
                              float* out_stats, cudaStream_t stream) {
  namespace ks = kps::score;
  const kps::NvtxRange range("kps_token_logprobs");
  ks::Args a = {};
  const kps_status st = ks::check(logits, dt, N, V, ld, tokens, temperature, temperatures, &a);
  if (st != KPS_OK) return st;
  if (n < 0 || n > 1024 || n > V) return KPS_ERR_INVALID_ARG;
  if (N == 0) return KPS_OK;
  if (n > 0 && (!out_ids || !out_logprobs)) return KPS_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(out_logprob), static_cast<const void*>(out_entropy),
                        static_cast<const void*>(out_rank), static_cast<const void*>(out_ids),
                        static_cast<const void*>(out_logprobs), static_cast<const void*>(out_stats)})
    if (ks::misaligned(p, 4)) return KPS_ERR_INVALID_ARG;
  a.n = static_cast<int>(n);
  a.logprob = out_logprob;
  a.entropy = out_entropy;
  a.rank = out_rank;
  a.ids = out_ids;
  a.logprobs = out_logprobs;
  if (out_stats) {
    a.max = out_stats;
    a.eps = out_stats + N;
    a.q = out_stats + 2 * N;
  }
  return ks::launch_score(a, dt, stream);
}

kps_status kps_token_logprobs_backward(const void* logits, kps_dtype dt, int64_t N, int64_t V, int64_t ld,
                                       const int64_t* tokens, float temperature, const float* temperatures,
                                       const float* grad_logprob, const float* grad_entropy, const float* stats,
                                       void* out_grad, int64_t ld_grad, cudaStream_t stream) {
  namespace ks = kps::score;
  const kps::NvtxRange range("kps_token_logprobs_backward");
  ks::Grad P = {};
  kps_status st = ks::check(logits, dt, N, V, ld, tokens, temperature, temperatures, &P.a);
  if (st != KPS_OK || N == 0) return st;
  if (!stats || ks::misaligned(stats, 4) || ks::misaligned(grad_logprob, 4) || ks::misaligned(grad_entropy, 4))
    return KPS_ERR_INVALID_ARG;
  if ((st = kps::check_grad(logits, N, V, ld, dt, out_grad, ld_grad)) != KPS_OK) return st;
  P.a.max = const_cast<float*>(stats);
  P.a.eps = P.a.max + N;
  P.a.q = P.a.max + 2 * N;
  P.g = grad_logprob;
  P.h = grad_entropy;
  P.out = out_grad;
  P.ld_out = ld_grad;
  return ks::launch_slope<false>(P, dt, stream);
}

kps_status kps_policy_loss_grad(const void* logits, kps_dtype dt, int64_t N, int64_t V, int64_t ld, const int64_t* tokens,
                                float temperature, const float* temperatures, const float* old_logprob,
                                const float* advantage, const float* ref_logprob, const float* weight, float clip_low,
                                float clip_high, float kl_coef, float entropy_coef, float* out_loss, float* out_logprob,
                                float* out_entropy, void* out_grad, int64_t ld_grad, cudaStream_t stream) {
  namespace ks = kps::score;
  const kps::NvtxRange range("kps_policy_loss_grad");
  ks::Grad P = {};
  kps_status st = ks::check(logits, dt, N, V, ld, tokens, temperature, temperatures, &P.a);
  if (st != KPS_OK) return st;
  if (!(clip_low >= 0.0f) || !(clip_high >= 0.0f) || !std::isfinite(kl_coef) || !std::isfinite(entropy_coef)) return KPS_ERR_INVALID_ARG;
  if (N == 0) return KPS_OK;
  if (!old_logprob || !advantage || (kl_coef != 0.0f && !ref_logprob) || !out_loss || !out_logprob || !out_entropy)
    return KPS_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(old_logprob), static_cast<const void*>(advantage),
                        static_cast<const void*>(ref_logprob), static_cast<const void*>(weight),
                        static_cast<const void*>(out_loss), static_cast<const void*>(out_logprob),
                        static_cast<const void*>(out_entropy)})
    if (ks::misaligned(p, 4)) return KPS_ERR_INVALID_ARG;
  if ((st = kps::check_grad(logits, N, V, ld, dt, out_grad, ld_grad)) != KPS_OK) return st;
  P.a.weight = weight;
  P.old = old_logprob;
  P.advantage = advantage;
  P.ref = ref_logprob;
  P.lo = clip_low;
  P.hi = clip_high;
  P.kl = kl_coef;
  P.ent = entropy_coef;
  P.loss = out_loss;
  P.out = out_grad;
  P.ld_out = ld_grad;
  P.a.logprob = out_logprob;
  P.a.entropy = out_entropy;
  return dt == KPS_BF16 ? ks::launch_policy<true>(P, stream) : ks::launch_policy<false>(P, stream);
}

}  // extern "C"
