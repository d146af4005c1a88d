// kps_score.cuh — a row of logits as a distribution over its tokens: the largest logit, the sum of
// exponentials beside it and their first moment, from which the log-probability of a token, the
// entropy and both gradients follow.  Shared by the kernels that score given tokens and train on them.
//
// Per row, with T the temperature, m the largest logit and d_v = (x_v - m) / T <= 0:
//
//   eps = sum over all but one element equal to m of exp(d_v),     S = 1 + eps
//   Q   = sum_v exp(d_v) (-d_v) / S
//   logprob_t = d_t - ln(1 + eps)            entropy = ln(1 + eps) + Q
//   d logprob_t / d x_v = (delta_tv - p_v) / T           1 - p_t = eps / S where x_t = m
//   d entropy   / d x_v = -p_v (d_v + Q) / T
//
// The largest element stays out of the sum, so that rows which are all but certain (most rows of a
// trained model) keep the relative precision of what is small in them: every sum above has terms of
// one sign, and no result is a difference of two larger ones.
#pragma once

#include "kps.h"
#include "kps_stream.cuh"

#include <cmath>

namespace kps {
namespace score {

using namespace stream;

constexpr int64_t kMaxV = 1 << 20;

// What scoring needs and gives; the outputs that are not wanted are nullptr.
struct Args {
  const void* x;
  int64_t N, ld;
  int V, n;            // n alternatives
  float tau;           // where taus is nullptr
  const float* taus;
  const int64_t* tokens;
  const float* weight;  // a row of weight 0 is empty, or nullptr (without alternatives only)
  float* logprob;
  float* entropy;
  int32_t* rank;
  int32_t* ids;        // [N, n]
  float* logprobs;     // [N, n]
  float *max, *eps, *q;  // [N] each: m, eps, Q
};

// Scoring with alternatives (kps_top.cu).
kps_status launch_alternatives(const Args& a, kps_dtype dt, cudaStream_t stream);

// A temperature of a row that is no positive normal number (the rows that the sampling step takes
// greedily) counts as 1.
__device__ __forceinline__ float row_tau(const float* taus, float tau, int64_t row) {
  if (!taus) return tau;
  const float t = taus[row];
  return t >= FLT_MIN && t < INFINITY ? t : 1.0f;
}

// (x - m) / tau, also where the difference of the two leaves fp32.
__device__ __forceinline__ float scaled(float x, float m, float tau) {
  const float d = x - m;
  return fabsf(d) < INFINITY ? d / tau : (0.5f * x - 0.5f * m) / (0.5f * tau);
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// No exponent goes below this: 2^z is zero long before, and 0 z stays a number (masks of -inf and of
// the type's lowest value).
constexpr float kFloor = -1024.0f;
__device__ __forceinline__ float exponent(float x, float ref, float c) { return max_nan((x - ref) * c, kFloor); }

// S = sum 2^z and W = sum 2^z z over elements with z = (x - ref) c <= 0.  The difference comes first, so that
// equal logits have equal exponents and small ones their own precision (a multiply-add of x would leave the
// rounding of ref c in them).  (Clamping bf16 logits two at a time instead of exponents: 2% slower.)
// kFree: no exponent is below kFloor.
template <bool kBF16>
struct Moments {
  f32x2 s[2] = {0ull, 0ull}, w[2] = {0ull, 0ull};
  template <bool kFree = false>
  __device__ __forceinline__ void add(const uint4& v, f32x2 nref2, f32x2 c2) {
#pragma unroll
    for (int i = 0; i < (kBF16 ? 4 : 2); ++i) {
      float a, b;
      unpack2(mul2(add2(pair_of<kBF16>(v, i), nref2), c2), a, b);
      if (!kFree) {
        a = max_nan(a, kFloor);
        b = max_nan(b, kFloor);
      }
      const f32x2 e = pack2(ex2(a), ex2(b));
      s[i & 1] = add2(s[i & 1], e);
      w[i & 1] = fma2(e, pack2(a, b), w[i & 1]);
    }
  }
  // The reference moves up by delta exponents.
  __device__ __forceinline__ void shift(float delta) {
    const float f = ex2(-delta);
    const f32x2 nd = pack2(-delta, -delta), f2 = pack2(f, f);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      w[i] = mul2(f2, fma2(s[i], nd, w[i]));
      s[i] = mul2(f2, s[i]);
    }
  }
  __device__ __forceinline__ float sum() const {
    float a, b;
    unpack2(add2(s[0], s[1]), a, b);
    return a + b;
  }
  __device__ __forceinline__ float moment() const {
    float a, b;
    unpack2(add2(w[0], w[1]), a, b);
    return a + b;
  }
};

// The larger, or the smaller, of two vectors element by element (NaN ignored).
template <bool kBF16, bool kMin = false>
__device__ __forceinline__ uint4 vec_extreme(const uint4& v, const uint4& w) {
  auto of = [](uint32_t a, uint32_t b) -> uint32_t {
    if (kBF16) {
      const __nv_bfloat162 x = reinterpret_cast<const __nv_bfloat162&>(a), y = reinterpret_cast<const __nv_bfloat162&>(b);
      const __nv_bfloat162 m = kMin ? __hmin2(x, y) : __hmax2(x, y);
      return reinterpret_cast<const uint32_t&>(m);
    }
    const float x = __uint_as_float(a), y = __uint_as_float(b);
    return __float_as_uint(kMin ? fminf(x, y) : fmaxf(x, y));
  };
  return make_uint4(of(v.x, w.x), of(v.y, w.y), of(v.z, w.z), of(v.w, w.w));
}
// The smallest element of a vector (NaN ignored).
template <bool kBF16>
__device__ __forceinline__ float vec_min(const uint4& w) {
  const uint32_t sign = kBF16 ? 0x80008000u : 0x80000000u;
  return -vec_max<kBF16>(make_uint4(w.x ^ sign, w.y ^ sign, w.z ^ sign, w.w ^ sign));
}

// Takes the first element equal to m out of a vector.
template <bool kBF16>
__device__ __forceinline__ void strike(uint4& v, float m) {
  uint32_t word[4] = {v.x, v.y, v.z, v.w};
  bool found = false;
#pragma unroll
  for (int e = 0; e < (kBF16 ? 8 : 4); ++e) {
    const float y = kBF16 ? __uint_as_float((e & 1) ? (word[e / 2] & 0xFFFF0000u) : (word[e / 2] << 16)) : __uint_as_float(word[e]);
    if (found || y != m) continue;
    found = true;
    if (kBF16) word[e / 2] = (e & 1) ? (word[e / 2] & 0x0000FFFFu) | 0xFF800000u : (word[e / 2] & 0xFFFF0000u) | 0x0000FF80u;
    else word[e] = 0xFF800000u;
  }
  v = make_uint4(word[0], word[1], word[2], word[3]);
}

// How many elements of a vector are larger than y (a value of the row's type).
template <bool kBF16>
__device__ __forceinline__ float count_above(const uint4& v, float y) {
  if (kBF16) {
    const __nv_bfloat162 t = __float2bfloat162_rn(y);
    auto above = [&](uint32_t w) { return __hgt2(reinterpret_cast<const __nv_bfloat162&>(w), t); };
    const float2 n = __bfloat1622float2(__hadd2(__hadd2(above(v.x), above(v.y)), __hadd2(above(v.z), above(v.w))));
    return n.x + n.y;
  }
  return (__uint_as_float(v.x) > y ? 1.0f : 0.0f) + (__uint_as_float(v.y) > y ? 1.0f : 0.0f) +
         (__uint_as_float(v.z) > y ? 1.0f : 0.0f) + (__uint_as_float(v.w) > y ? 1.0f : 0.0f);
}

// A part of a row: its largest logit, S and W of everything in it but one element equal to that
// (against it), and how many of its elements are larger than the token's.
struct Part {
  float m, s, w, above;
};

// What a part adds to the sums of a row whose largest logit is m; `own`: the part whose largest
// element stands for the row's.
__device__ __forceinline__ void part_to_row(const Part& p, bool own, float m, float c, float& s, float& w) {
  if (p.m == -INFINITY) {  // nothing finite: zeros, or NaN
    s = p.s;
    w = p.w;
    return;
  }
  const float all = own ? p.s : p.s + 1.0f;
  const float delta = fminf((m - p.m) * c, -kFloor), f = ex2(-delta);  // (NaN: the row has none of this anyway)
  s = f * all;
  w = f * (p.w - delta * all);
}

// The statistics of a row: m, eps, Q; ok: it has a distribution.
struct Row {
  float m, eps, q;
  bool ok;
  __device__ __forceinline__ Row(float m_, float s, float w) {
    m = m_;
    eps = s;
    q = -kLn2 * w / (1.0f + s);
    ok = fabsf(m) < INFINITY && s < INFINITY && q < INFINITY;  // (NaN fails too)
    if (!ok) m = eps = q = NAN;
  }
  __device__ __forceinline__ Row(const float* pm, const float* pe, const float* pq, int64_t row) : m(pm[row]), eps(pe[row]), q(pq[row]) {
    ok = m == m;
  }
  __device__ __forceinline__ float logprob(float x, float tau) const { return ok ? scaled(x, m, tau) - log1pf(eps) : NAN; }
  __device__ __forceinline__ float entropy() const { return log1pf(eps) + q; }
};

__device__ __forceinline__ float no_nan(float x) { return isnan(x) ? -INFINITY : x; }

// Writes a row's results, by one thread.
__device__ __forceinline__ void put_row(const Args& a, int64_t row, const Row& r, float token, float tau, float above) {
  if (a.logprob) a.logprob[row] = r.logprob(token, tau);
  if (a.entropy) a.entropy[row] = r.entropy();
  if (a.rank) a.rank[row] = static_cast<int32_t>(above);
  if (a.max) {
    a.max[row] = r.m;
    a.eps[row] = r.eps;
    a.q[row] = r.q;
  }
}
// An empty row, by the whole block.
__device__ __forceinline__ void put_empty(const Args& a, int64_t row, int threads) {
  for (int i = threadIdx.x; i < a.n; i += threads) {
    a.ids[row * a.n + i] = -1;
    a.logprobs[row * a.n + i] = -INFINITY;
  }
  if (threadIdx.x == 0) {
    if (a.logprob) a.logprob[row] = 0.0f;
    if (a.entropy) a.entropy[row] = 0.0f;
    if (a.rank) a.rank[row] = -1;
    if (a.max) a.max[row] = a.eps[row] = a.q[row] = 0.0f;
  }
}

}  // namespace score
}  // namespace kps
