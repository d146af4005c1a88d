// kps_top.cu — the top logits of every row with the log-sum-exps that turn them into
// log-probabilities: what serving returns beside a sampled token, and what a teacher hands to
// the distillation loss.
//
// Per row, with the order "value descending, index ascending" (NaN counts as -inf) and a = x / tau:
//
//   ids, values = the first n elements of the order       lse  = ln sum_v exp(a_v)
//   rest = ln sum_{v not among them} exp(a_v)             logprob = a_token - lse
//
// One pass over the row.  A threshold from a sample of 2048 elements is reached by a few times n
// elements; those go to a list in shared memory, all others into a running sum of exponentials.
// The list is sorted, its first n are the top, and what is left of it joins the sum: the rest is
// a sum of its own, never a difference of two large ones.  A list that came out too short or too
// long (the sample misjudged the row, or ties crowd the threshold) sends the row to an exact
// selection by digits.

#include "kps.h"
#include "kps_host.h"
#include "kps_stream.cuh"

#include <cooperative_groups.h>

#include <climits>
#include <cmath>

namespace cg = cooperative_groups;

namespace kps {
namespace top {

using namespace stream;

constexpr int kNT = 256;  // threads per CTA
constexpr int kNW = kNT / 32;
constexpr int kU = 4;          // 16-byte loads each thread keeps in flight
constexpr int kMaxN = 1024;    // the framework's top-k limit
constexpr int64_t kMaxV = 1 << 20;
constexpr int kMaxCS = 8;      // widest cluster (the portable limit)
constexpr int kCap = 4096;     // list entries
constexpr int kPer = 8;        // sampled elements per thread
constexpr int kSamp = kNT * kPer;
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;

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

struct Smem {
  unsigned long long list[kCap];
  uint32_t hist[256];
  float red[kNW][2];
  float part[kMaxCS][2];     // the sums of the cluster's CTAs
  uint32_t count[kMaxCS];    // their list lengths
  uint32_t n_list;
  uint32_t found;
  int nan;
};

__device__ __forceinline__ Sum2 block_merge(Sum2 v, float c, float (*red)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = warp_merge(v, c);
  __syncthreads();
  if (lane == 0) {
    red[warp][0] = v.ref;
    red[warp][1] = v.s;
  }
  __syncthreads();
  v.ref = red[lane & (kNW - 1)][0];
  v.s = lane < kNW ? red[lane][1] : 0.0f;
  return warp_merge(v, c);
}
__device__ __forceinline__ void add_one(Sum2& sum, float x, float c) {
  if (x > sum.ref + kRaise / c) sum.raise(clamp_ref(x), c);
  sum.s += ex2((x - sum.ref) * c);
}

// The largest key (its low 16 bits zero) that at least r of the block's sampled keys reach.
__device__ __forceinline__ uint32_t sample_threshold(const uint32_t (&key)[kPer], uint32_t r, Smem& sm) {
  uint32_t t = 0;
  for (int bit = 31; bit >= 16; --bit) {
    const uint32_t mid = t | (1u << bit);
    uint32_t n = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) n += key[i] >= mid ? 1u : 0u;
    n = __reduce_add_sync(0xffffffffu, n);
    uint32_t* slot = &sm.hist[bit];  // one counter per round, zeroed beforehand
    if ((threadIdx.x & 31) == 0) atomicAdd(slot, n);
    __syncthreads();
    if (*slot >= r) t = mid;
  }
  return t;
}

// Descending bitonic sort of list[0..N), N a power of two.
__device__ __forceinline__ void sort_desc(unsigned long long* a, int N) {
  for (int k = 2; k <= N; k <<= 1) {
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int t = threadIdx.x; t < N / 2; t += kNT) {
        const int i = 2 * t - (t & (j - 1)), l = i + j;
        const unsigned long long p = a[i], q = a[l];
        if (((i & k) == 0) ? p < q : p > q) {
          a[i] = q;
          a[l] = p;
        }
      }
      __syncthreads();
    }
  }
}

// One element at a time over the row: f(value with NaN -> -inf, index).
template <bool kBF16, class F>
__device__ __forceinline__ void each(const RowView<kBF16>& x, F&& f) {
  for (int v = threadIdx.x; v < x.V; v += kNT) f(clean(x.at(v)), v);
}

// The exact selection, by one CTA: the n-th element of the order by 8-bit digits of its key and,
// among equal keys, of its index; then the list of the n elements and the sum of all others.
template <bool kBF16>
__device__ __noinline__ Sum2 exact_select(const RowView<kBF16>& x, int n, float c, Smem& sm) {
  uint32_t need = static_cast<uint32_t>(n);
  unsigned long long at = 0;  // the digits found so far, from the top of the 64-bit word
  if (n > 0) {
    for (int shift = 56; shift >= 0; shift -= 8) {
      if (shift == 24) {  // indexes are below 2^20, their complements share the top 12 bits
        at |= 0xFFull << 24;
        continue;
      }
      for (int i = threadIdx.x; i < 256; i += kNT) sm.hist[i] = 0u;
      __syncthreads();
      each<kBF16>(x, [&](float y, int v) {
        const unsigned long long w = word_of(fkey(y), v);
        if (shift == 56 || (w >> (shift + 8)) == (at >> (shift + 8))) atomicAdd(&sm.hist[(w >> shift) & 255u], 1u);
      });
      __syncthreads();
      if (threadIdx.x == 0) {
        uint32_t above = 0, d = 255;
        while (d > 0 && above + sm.hist[d] < need) above += sm.hist[d--];
        sm.found = d;
        sm.n_list = above;
      }
      __syncthreads();
      at |= static_cast<unsigned long long>(sm.found) << shift;
      need -= sm.n_list;
      __syncthreads();
    }
  }
  if (threadIdx.x == 0) sm.n_list = 0u;
  __syncthreads();
  Sum2 sum{-FLT_MAX, 0.0f};
  each<kBF16>(x, [&](float y, int v) {
    const unsigned long long w = word_of(fkey(y), v);
    if (n > 0 && w >= at) {
      sm.list[atomicAdd(&sm.n_list, 1u)] = w;  // n of them
    } else {
      add_one(sum, y, c);
    }
  });
  return block_merge(sum, c, sm.red);
}

template <bool kBF16>
__global__ void __launch_bounds__(kNT) top_kernel(const Params P) {
  constexpr int G = kBF16 ? 8 : 4;
  extern __shared__ __align__(16) unsigned char smem[];
  Smem& sm = *reinterpret_cast<Smem*>(smem);
  const int CS = static_cast<int>(cg::this_cluster().num_blocks());
  const int rank = static_cast<int>(cg::this_cluster().block_rank());
  const int64_t row = blockIdx.x / CS;
  const int n = P.n;
  const float c = P.c;
  const RowView<kBF16> x(P.x, row * P.ld, P.V);
  const int g0 = static_cast<int>(static_cast<int64_t>(x.nv) * rank / CS);
  const int g1 = static_cast<int>(static_cast<int64_t>(x.nv) * (rank + 1) / CS);
  // every CTA of the cluster runs before any writes into another's shared memory
  if (CS > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

  // ---- the threshold: every CTA of the row takes the same sample --------------------------
  float thr = INFINITY;  // n == 0: nothing is listed
  if (n > 0) {
    // kSamp places spread over the row (all of it when it is that short), each the largest of
    // `m` elements for the longest rows
    const int m = (P.V + (1 << 18) - 1) >> 18;
    uint32_t key[kPer];
    float y[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int s = i * kNT + static_cast<int>(threadIdx.x);
      // runs of 32 consecutive elements
      const int64_t v = P.V <= kSamp ? s : static_cast<int64_t>(s >> 5) * (P.V - 32 * m) / (kSamp / 32 - 1) + (s & 31);
      y[i] = v < P.V ? x.at(static_cast<int>(v)) : -INFINITY;
      for (int j = 1; j < m; ++j) y[i] = fmaxf(y[i], x.at(static_cast<int>(v) + 32 * j));
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) key[i] = fkey(clean(y[i]));
    for (int i = threadIdx.x; i < 256; i += kNT) sm.hist[i] = 0u;
    if (threadIdx.x == 0) {
      sm.n_list = 0u;
      sm.nan = 0;
    }
    __syncthreads();
    // the number of row elements that reach the r-th largest of the sample is about r times
    // `one`, give or take sqrt(r) times `one`: four of these on the safe side
    const float one = fmaxf(1.0f, static_cast<float>(P.V) / static_cast<float>(kSamp * m));
    const float r = static_cast<float>(n) / one;
    const uint32_t want = static_cast<uint32_t>(r + (P.V <= kSamp ? 0.0f : 4.0f * sqrtf(r) + 6.0f));
    const uint32_t t = want >= static_cast<uint32_t>(kSamp) ? 0u : sample_threshold(key, want < 1u ? 1u : want, sm);
    thr = t <= kKeyNegInf ? -INFINITY : kfloat(t);
  } else {
    if (threadIdx.x == 0) {
      sm.n_list = 0u;
      sm.nan = 0;
    }
    __syncthreads();
  }

  // ---- the pass -----------------------------------------------------------------------------
  Sum2 sum{-FLT_MAX, 0.0f};
  const float lift = kRaise / c;
  auto put = [&](float y, int v) {
    const uint32_t pos = atomicAdd(&sm.n_list, 1u);
    if (pos < static_cast<uint32_t>(kCap)) sm.list[pos] = word_of(fkey(y + 0.0f), v);
  };
  for (int base = g0; base < g1; base += kNT * kU) {
    uint4 w[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int g = base + u * kNT + static_cast<int>(threadIdx.x);
      w[u] = g < g1 ? ld_stream(x.vec + g) : neg_inf_vec<kBF16>();
    }
    float mx = -INFINITY;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int g = base + u * kNT + static_cast<int>(threadIdx.x);
      float m = vec_max<kBF16>(w[u]);
      if (m >= thr && g < g1) {
        uint32_t word[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
        const int v0 = x.head + g * G;
#pragma unroll
        for (int e = 0; e < G; ++e) {
          const float y = kBF16 ? __uint_as_float((e & 1) ? (word[e / 2] & 0xFFFF0000u) : (word[e / 2] << 16))
                                : __uint_as_float(word[e]);
          if (y >= thr) {
            put(y, v0 + e);
            if (kBF16) word[e / 2] = (e & 1) ? (word[e / 2] & 0x0000FFFFu) | 0xFF800000u : (word[e / 2] & 0xFFFF0000u) | 0x0000FF80u;
            else word[e] = 0xFF800000u;
          }
        }
        w[u] = make_uint4(word[0], word[1], word[2], word[3]);
        m = vec_max<kBF16>(w[u]);
      }
      mx = fmaxf(mx, m);
    }
    if (mx > sum.ref + lift) sum.raise(clamp_ref(mx), c);
#pragma unroll
    for (int u = 0; u < kU; ++u) add_vec<kBF16>(sum, w[u], c);
  }
  // the elements outside the vectors: the head with rank 0, the tail with the last rank
  if (static_cast<int>(threadIdx.x) < x.loose()) {
    const int v = x.loose_at(threadIdx.x);
    if ((v < x.head) ? rank == 0 : rank == CS - 1) {
      const float y = x.at(v);
      if (y >= thr) put(y, v);
      else add_one(sum, y, c);
    }
  }
  sum = block_merge(sum, c, sm.red);  // its barriers publish the list

  // ---- rank 0 gathers the lists and the sums --------------------------------------------------
  uint32_t count = sm.n_list;
  if (CS > 1) {
    cg::cluster_group cl = cg::this_cluster();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (threadIdx.x == 0) {
      float* to = cl.map_shared_rank(&sm.part[rank][0], 0);
      to[0] = sum.ref;
      to[1] = sum.s;
      *cl.map_shared_rank(&sm.count[rank], 0) = count;
    }
    cl.sync();
    if (rank == 0) {
      count = 0;
      for (int q = 0; q < CS; ++q) {
        const uint32_t nq = sm.count[q];
        if (q > 0) {
          sum = merge(sum, Sum2{sm.part[q][0], sm.part[q][1]}, c);
          const unsigned long long* from = cl.map_shared_rank(&sm.list[0], q);
          if (count + nq <= static_cast<uint32_t>(kCap))
            for (uint32_t i = threadIdx.x; i < nq; i += kNT) sm.list[count + i] = from[i];
        }
        count = nq > static_cast<uint32_t>(kCap) || count > static_cast<uint32_t>(kCap) ? kCap + 1u : count + nq;
      }
    }
    cl.sync();  // the other CTAs' lists are read
    if (rank != 0) return;
  }

  // a NaN anywhere in the sum, or a list of the wrong length: the exact selection
  if (isnan(sum.s) || count < static_cast<uint32_t>(n) || count > static_cast<uint32_t>(kCap)) {
    sum = exact_select<kBF16>(x, n, c, sm);
    count = static_cast<uint32_t>(n);
  }
  int N = 2;
  while (N < static_cast<int>(count)) N <<= 1;
  for (int i = static_cast<int>(count + threadIdx.x); i < N; i += kNT) sm.list[i] = 0ull;  // below every word
  __syncthreads();
  if (n > 0) sort_desc(sm.list, N);

  // ---- the outputs ----------------------------------------------------------------------------
  Sum2 lead{-FLT_MAX, 0.0f}, left{-FLT_MAX, 0.0f};  // of the top, and of the list behind it
  for (int i = threadIdx.x; i < static_cast<int>(count); i += kNT) {
    const unsigned long long w = sm.list[i];
    const float y = word_value(w);
    add_one(i < n ? lead : left, y, c);
    if (i < n) {
      P.ids[row * n + i] = word_index(w);
      P.values[row * n + i] = y;
    }
  }
  left = block_merge(left, c, sm.red);
  sum = merge(sum, left, c);
  lead = block_merge(lead, c, sm.red);
  if (threadIdx.x == 0) {
    const Sum2 all = merge(lead, sum, c);
    // a sum of nothing is -inf; a sum with +inf in it is +inf
    auto ln = [&](const Sum2& s) { return s.s == 0.0f ? -INFINITY : logf(s.s) + s.ref / P.tau; };
    const float lse = ln(all);
    if (P.lse) P.lse[row] = lse;
    if (P.rest) P.rest[row] = ln(sum);
    if (P.logprob) {
      const int64_t t = P.tokens[row];
      // relative to the sum's reference: lse and the token's logit are both large
      float lp = -INFINITY;
      if (t >= 0 && t < P.V) {
        const float y = clean(x.at(static_cast<int>(t)));
        lp = isinf(lse) ? y / P.tau - lse : (y - all.ref) / P.tau - logf(all.s);
      }
      P.logprob[row] = lp;
    }
  }
}

// ------------------------------------------------------------------------------------------
// Host side
// ------------------------------------------------------------------------------------------
template <bool kBF16>
static kps_status launch(const Params& P, cudaStream_t stream) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
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
  lc.dynamicSmemBytes = sizeof(Smem);
  lc.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  if (cudaLaunchKernelEx(&lc, top_kernel<kBF16>, P) != cudaSuccess) {
    (void)cudaGetLastError();
    return KPS_ERR_CUDA;
  }
  return KPS_OK;
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
