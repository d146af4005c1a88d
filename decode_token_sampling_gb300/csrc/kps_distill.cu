// kps_distill.cu — the distillation loss of a student's rows of logits against the top logits
// of a teacher, and its gradient.
//
// Per row, with tau the temperature, (id_k, t_k) the teacher's slots and, optionally, r the
// log-sum-exp of everything the teacher's list leaves out:
//
//   p   = softmax([t_k / tau ..., r])                        over the valid slots and the rest
//   L   = ln sum_v exp(s_v / tau)                            over the student's whole row
//   R   = ln sum_{v not in the list} exp(s_v / tau)
//   loss = w tau^2 (sum_k p_k (ln p_k - s_{id_k} / tau + L) + p_r (ln p_r - R + L))
//   d loss / d s_v = w tau (exp(s_v / tau - L) - sum_{k: id_k = v} p_k)        v in the list
//                    w tau (exp(s_v / tau - L) - p_r exp(s_v / tau - R))       else
//
// The work is one pass over the student's row for the loss (V elements read) and one more for
// the gradient (V read, V written): both are bound by memory.  Every exponential is taken of a
// difference to a reference logit, and the loss is assembled from quantities relative to the
// largest student logit among the list's tokens and to the teacher's largest value, so nothing
// of the size of L itself is ever subtracted.

#include "kps.h"
#include "kps_host.h"
#include "kps_stream.cuh"

#include <cooperative_groups.h>

#include <atomic>
#include <cfloat>
#include <climits>
#include <cmath>

namespace cg = cooperative_groups;

namespace kps {
namespace distill {

using namespace stream;

constexpr int kNT = 256;  // threads per CTA
constexpr int kNW = kNT / 32;
// 16-byte loads each thread keeps in flight, and the CTAs an SM then holds.  The forward with eight
// and four takes 154 us for 4096 rows of 151936 bf16 (a quarter masked) and 49.4 us for 1024 of
// 128256, with six and five 153 and 53.2 us, with four and five 164 and 55.9 us; the backward of the
// latter with six and five 86.8 us, with eight and four 88.6 us, with four and five 87.6 us.
template <int kMode>
struct Flight {
  static constexpr int loads = kMode == 0 ? 8 : 6, ctas = kMode == 0 ? 4 : 5;
};
constexpr int kMaxK = 1024;   // teacher slots a row may have (the framework's top-k limit)
constexpr int64_t kMaxV = 1 << 20;
constexpr int kMaxCS = 8;     // widest cluster (the portable limit)
constexpr int kMaxDevices = 64;
constexpr int kStats = 4;     // floats of statistics per row

enum Mode { kForward = 0, kBackward = 1, kBoth = 2 };

struct Params {
  const void* student;
  int64_t N, ld;
  int V, K;
  const int32_t* ids;
  const void* values;
  int values_bf16;
  const float* rest;     // or nullptr
  const float* weight;   // or nullptr: 1
  float tau, c, c_lo;    // c + c_lo = log2(e) / tau
  const float* upstream; // gradient modes: the loss's gradient per row, or nullptr: 1
  float* loss;           // [N] (kForward, kBoth)
  float* stats;          // [N, kStats]: written by kForward (may be nullptr), read by kBackward
  void* grad;
  int64_t ld_grad;
};

// Shared memory: the teacher's slots, the hash table of the list's distinct tokens and, for the
// student's sum, the bitmap of the list's tokens in this CTA's part of the row.
struct Layout {
  size_t id, e, v, hash, bits, total;
  int hash_size;
};
__host__ __device__ inline Layout make_layout(int K, int64_t chunk, bool bitmap) {
  Layout L;
  size_t off = 0;
  const size_t k4 = (static_cast<size_t>(K) * 4 + 15) / 16 * 16;
  L.id = off; off += k4;
  L.e = off;  off += k4;
  L.v = off;  off += k4;
  L.hash_size = 32;
  while (L.hash_size < 2 * K) L.hash_size *= 2;
  L.hash = off;
  off += static_cast<size_t>(L.hash_size) * 4;
  L.bits = off;
  if (bitmap) off += (static_cast<size_t>(chunk) + 31) / 32 * 4 / 16 * 16 + 32;
  L.total = off;
  return L;
}

__device__ __forceinline__ float teacher_value(const Params& P, int64_t i) {
  return P.values_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(P.values)[i])
                       : static_cast<const float*>(P.values)[i];
}

// The block's sum; every thread gets it.
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
  if ((x - sum.ref) * c > kRaise) sum.raise(clamp_ref(x), c);
  sum.s += ex2((x - sum.ref) * c);
}

// ---- the list, to more than fp32's rounding of its exponents ----------------------------------
//
// The gradient of a list's token is a difference of two masses, and the loss a sum of terms that
// cancel when the student comes near its teacher: there the rounding of an exponent of 20 or 30
// would show.  Exponents of the list's tokens and of the rest are therefore carried as two floats
// (the sum over the row needs none of that: its terms weigh little where their exponents are large).

// h + l = x - y exactly (Knuth's two-sum; l = 0 where the difference is not finite).
__device__ __forceinline__ void two_diff(float x, float y, float& h, float& l) {
  h = x - y;
  const float b = h - x;
  l = (x - (h - b)) + (-y - b);
  if (!(fabsf(h) < INFINITY)) l = 0.0f;
}
// 2^(h + l) for a small l.
__device__ __forceinline__ float ex2_two(float h, float l) {
  const float e = ex2(h);
  return l != 0.0f ? fmaf(e, l * kLn2, e) : e;
}
// 2^((x - ref) (c + c_lo)).
__device__ __forceinline__ float mass(float x, float ref, float c, float c_lo) {
  float h, l;
  two_diff(x, ref, h, l);
  const float z = h * c;
  const float rest = fmaf(h, c, -z) + fmaf(h, c_lo, l * c);
  return ex2_two(z, fabsf(z) < 1e30f ? rest : 0.0f);
}

// A sum as two floats: h + l (each addition's rounding error by Knuth's two-sum).
struct F2 {
  float h, l;
  __device__ __forceinline__ void add(float x) {
    const float t = h + x, b = t - h;
    const float e = (h - (t - b)) + (x - b);
    h = t;
    l += fabsf(t) < INFINITY ? e : 0.0f;
  }
  __device__ __forceinline__ void add(const F2& o) {
    add(o.h);
    l += o.l;
  }
  __device__ __forceinline__ float value() const { return h + l; }
};
__device__ __forceinline__ F2 warp_sum_two(F2 v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v.add(F2{__shfl_xor_sync(0xffffffffu, v.h, o), __shfl_xor_sync(0xffffffffu, v.l, o)});
  return v;
}
// log2((a + b) / (c + d)) without the roundings of the sums and the quotient.
__device__ __forceinline__ float log2_ratio(F2 a, float b, F2 c, float d) {
  a.add(b);
  c.add(d);
  const float q = a.h / c.h;
  if (!(q > 0.0f && q < INFINITY)) return log2f(q);
  return log2f(q) + kLog2e * ((fmaf(-q, c.h, a.h) + a.l) / a.h - c.l / c.h);
}

// The teacher's side of a row against the reference tref: E = sum e_k, W = sum e_k (t_k - s_k) / kWScale,
// t_k and s_k the teacher's value and the student's logit from their references (scaled so that no sum
// of them overflows) and e_k = 2^(t_k c); the rest's e_r = 2^(uh + ul).
constexpr float kWScale = 4096.0f;
struct Teacher {
  F2 E, W;
  float er, uh, ul;
  template <bool kRest>
  __device__ __forceinline__ void rest(float r, float tref, float tau, float c, float c_lo) {
    er = uh = ul = 0.0f;
    if (!kRest || r == -INFINITY) return;
    if (!(fabsf(tref * c) < 0x1p40f)) {
      // floats this large lie 2^16 apart, and their exponents would overflow: the rest either is the
      // largest class or has no mass beside it
      er = r * tau < tref ? 0.0f : fabsf(r) < INFINITY ? 1.0f : NAN;
      return;
    }
    const float a = r * kLog2e, b = tref * c;  // r is in nats at the temperature
    const float al = fmaf(r, kLog2e, -a) + r * 1.92596303e-8f, bl = fmaf(tref, c, -b) + tref * c_lo;
    two_diff(a, b, uh, ul);
    if (fabsf(uh) < 1e30f) {
      // large logits leave a and b with coarse last places: the low parts are not small beside uh
      const float lo = ul + (al - bl), h = uh + lo, back = h - uh;
      ul = (uh - (h - back)) + (lo - back);
      uh = h;
    } else {
      ul = 0.0f;
    }
    er = ex2_two(uh, ul);
  }
};

// Whether the student's sum outside the list holds up: near its reference, or (a teacher whose rest
// has no mass) nothing beside the list's.
__device__ __forceinline__ bool precise(const Sum2& rest, const Sum2& list, float er) {
  return rest.s >= 0x1p-60f || (er == 0.0f && rest.s >= 0.0f && list.s >= 0.5f);
}

// The divergence times the temperature, over kWScale.  list (against ref), rest, all: the student's
// sums.  Distances between references stay in units of logits, scaled: in exponents of 2, or rounded
// up, those of the type's lowest value (a masked student) would leave fp32 where the loss does not.
__device__ __forceinline__ float divergence(const Teacher& t, float ref, const F2& list, const Sum2& rest,
                                            const Sum2& all, float tau, float c) {
  constexpr float kDown = 1.0f / kWScale;  // a power of 2: no rounding
  const float unit = tau * kLn2 * kDown, moved = (all.ref - ref) * kDown;  // of an exponent of 2
  const float E = t.E.value(), W = t.W.value();
  // (list and rest against one reference: their sum as two floats)
  const bool same = rest.ref == ref;
  const F2 head = same ? list : F2{all.s, 0.0f};
  const float tail = same ? rest.s : 0.0f;
  if (t.er == 0.0f) return W / E + unit * log2_ratio(head, tail, t.E, 0.0f) + moved;
  if (rest.s == 0.0f) return INFINITY;  // the teacher's rest has mass, the student's none
  const float Et = E + t.er, pr = t.er / Et;
  // D = (uh + ul) - log2 of the student's rest against ref, whole powers of two first
  const uint32_t bits = __float_as_uint(rest.s);
  const float k = static_cast<float>(static_cast<int>(bits >> 23) - 127);
  const float m = __uint_as_float((bits & 0x007FFFFFu) | 0x3F800000u);
  const float D = unit * (((t.uh - k) + t.ul) - log2f(m)) - (rest.ref - ref) * kDown;
  if (!(pr >= 0.5f)) return (W + t.er * D) / Et + unit * log2_ratio(head, tail, t.E, t.er) + moved;
  // most mass is the rest's: ln p_r and ln q_r from what they leave, so that two numbers near
  // zero are not differences of large ones
  const float S = list.value();
  float q = 0.0f;
  if (S > 0.0f) {
    const float s = log2f(S / rest.s), z = s + (ref - rest.ref) * c;
    q = z > 24.0f ? unit * s + (ref - rest.ref) * kDown : tau * kDown * log1pf(ex2(z));
  }
  return W / Et - E / Et * D - tau * kDown * log1pf(E / t.er) + q;
}

// The row's loss.
__device__ __forceinline__ float row_loss(const Params& P, const Teacher& T, float ref, const F2& list, const Sum2& rest,
                                          const Sum2& all, float w) {
  const bool ok = all.s > 0.0f && all.s < INFINITY;
  return ok ? w * P.tau * divergence(T, ref, list, rest, all, P.tau, P.c) * kWScale : NAN;
}

// Writes zeros to this CTA's part of a row of the gradient.
template <bool kBF16>
__device__ __forceinline__ void zero_row(void* grad, int64_t offset, int V, int rank, int CS) {
  const RowView<kBF16> o(grad, offset, V);
  const int o0 = static_cast<int>(static_cast<int64_t>(o.nv) * rank / CS);
  const int o1 = static_cast<int>(static_cast<int64_t>(o.nv) * (rank + 1) / CS);
  uint4* ov = const_cast<uint4*>(o.vec);
  for (int g = o0 + static_cast<int>(threadIdx.x); g < o1; g += kNT) __stcs(ov + g, make_uint4(0u, 0u, 0u, 0u));
  if (rank == 0 && static_cast<int>(threadIdx.x) < o.loose()) {
    const int v = o.loose_at(threadIdx.x);
    if (kBF16) reinterpret_cast<__nv_bfloat16*>(const_cast<unsigned char*>(o.base))[v] = __float2bfloat16(0.0f);
    else reinterpret_cast<float*>(const_cast<unsigned char*>(o.base))[v] = 0.0f;
  }
}

// Takes the list's tokens (bits m) out of a vector.
template <bool kBF16>
__device__ __forceinline__ void drop_listed(uint4& v, uint32_t m) {
  uint32_t word[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < (kBF16 ? 8 : 4); ++e) {
    if (!((m >> e) & 1u)) continue;
    if (kBF16) word[e / 2] = (e & 1) ? (word[e / 2] & 0x0000FFFFu) | 0xFF800000u : (word[e / 2] & 0xFFFF0000u) | 0x0000FF80u;
    else word[e] = 0xFF800000u;
  }
  v = make_uint4(word[0], word[1], word[2], word[3]);
}

// Inserts a token of the list into a table of its distinct tokens; true when it was there already.
__device__ __forceinline__ bool insert_token(int32_t* hash, int size, int32_t id) {
  uint32_t h = (static_cast<uint32_t>(id) * 2654435761u) & (size - 1);
  for (int i = 0; i < size; ++i) {  // at most K of the 2K places are taken: it ends long before
    const int32_t old = atomicCAS(&hash[h], -1, id);
    if (old == -1) return false;
    if (old == id) return true;
    h = (h + 1) & (size - 1);
  }
  return false;
}

// Whether the table holds a token.
__device__ __forceinline__ bool has_token(const int32_t* hash, int size, int32_t id) {
  uint32_t h = (static_cast<uint32_t>(id) * 2654435761u) & (size - 1);
  for (int i = 0; i < size && hash[h] != -1; ++i, h = (h + 1) & (size - 1))
    if (hash[h] == id) return true;
  return false;
}

// Keys of floats that order as they do, for maxima by integer atomics (NaN excluded).
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// ---- the teacher's slots of a row ---------------------------------------------------------------
struct Slot {
  int32_t id;
  float t;
};
__device__ __forceinline__ Slot read_slot(const Params& P, int64_t row, int k) {
  return Slot{P.ids[row * P.K + k], teacher_value(P, row * P.K + k)};
}
__device__ __forceinline__ Slot first_slot(const Params& P, int64_t row) {
  return static_cast<int>(threadIdx.x) < P.K ? read_slot(P, row, threadIdx.x) : Slot{-1, -INFINITY};
}
// Slots k = threadIdx.x, + kNT, ... (the first of them already loaded): ids (-1: empty), the
// teacher's values and the student's logits to shared memory, the distinct tokens to the table, the
// keys of both largest values to top[], flags[0] set where a slot is filled and flags[1] where a
// token has two; visit(k, id) for the filled ones.  Warps without slots do nothing.
template <class View, class Visit>
__device__ __forceinline__ void read_slots(const Params& P, int64_t row, const View& x, Slot slot, int32_t* s_id, float* s_e,
                                           float* s_v, int32_t* s_hash, int hash_size, uint32_t* top, int* flags,
                                           Visit&& visit) {
  const int K = P.K;
  if (static_cast<int>(threadIdx.x & ~31u) >= K) return;
  uint32_t tk = 0, sk = 0;
  for (int k = threadIdx.x; k < K;) {
    const int32_t id = slot.id < 0 || slot.id >= P.V || slot.t == -INFINITY ? -1 : slot.id;
    const float s = id >= 0 ? x.at(id) : 0.0f;
    s_id[k] = id;
    s_e[k] = slot.t;
    s_v[k] = s;
    if (id >= 0) {
      flags[0] = 1;
      if (!isnan(slot.t)) tk = max(tk, order_key(slot.t));
      if (!isnan(s)) sk = max(sk, order_key(s));
      if (insert_token(s_hash, hash_size, id)) flags[1] = 1;
      visit(k, id);
    }
    k += kNT;
    if (k < K) slot = read_slot(P, row, k);
  }
  __syncwarp();
  tk = __reduce_max_sync(0xffffffffu, tk);
  sk = __reduce_max_sync(0xffffffffu, sk);
  if ((threadIdx.x & 31) == 0) {
    atomicMax(&top[0], tk);
    atomicMax(&top[1], sk);
  }
}
// The references: the teacher's largest class (its rest in nats at tau included), and the largest
// student logit among the list's tokens (0 where all of them are -inf).
__device__ __forceinline__ float teacher_ref(const uint32_t* top, float r, float tau) {
  return clamp_ref(fmaxf(top[0] ? order_value(top[0]) : -INFINITY, r * tau));
}
__device__ __forceinline__ float student_ref(const uint32_t* top) {
  return top[1] > order_key(-INFINITY) ? clamp_ref(order_value(top[1])) : 0.0f;
}
// The slots' masses in the place of their values, and each warp's part of E, W and the student's sum
// over the list (its distinct tokens).
__device__ __forceinline__ void slot_masses(const Params& P, int K, float tref, float ref, bool dup, const int32_t* s_id,
                                            float* s_e, float* s_v, F2 (*sums)[3]) {
  if (static_cast<int>(threadIdx.x & ~31u) >= K) return;
  F2 E = {}, W = {}, S = {};
  for (int k = threadIdx.x; k < K; k += kNT) {
    const int32_t id = s_id[k];
    float e = 0.0f, q = 0.0f;
    if (id >= 0) {
      const float t = s_e[k], sv = s_v[k];
      e = mass(t, tref, P.c, P.c_lo);
      q = mass(sv, ref, P.c, P.c_lo);
      E.add(e);
      if (e != 0.0f) W.add(e * (((t - tref) - (sv - ref)) * (1.0f / kWScale)));  // NaN stays (e is NaN then)
      bool first = true;  // a token of several slots counts once
      if (dup)
        for (int j = 0; j < k; ++j) first = first && s_id[j] != id;
      if (first) S.add(q);
    }
    s_e[k] = e;
    s_v[k] = q;
  }
  __syncwarp();
  E = warp_sum_two(E);
  W = warp_sum_two(W);
  S = warp_sum_two(S);
  if ((threadIdx.x & 31) == 0) {
    F2* to = sums[threadIdx.x >> 5];
    to[0] = E;
    to[1] = W;
    to[2] = S;
  }
}
// All of that, after a barrier; returns the student's sum over the list.
template <bool kRest>
__device__ __forceinline__ F2 collect(const F2 (*sums)[3], int K, float r, float tref, float tau, float c, float c_lo,
                                      Teacher& T) {
  T = Teacher{};
  F2 S = {};
  for (int i = 0; i < kNW && i * 32 < K; ++i) {
    T.E.add(sums[i][0]);
    T.W.add(sums[i][1]);
    S.add(sums[i][2]);
  }
  T.rest<kRest>(r, tref, tau, c, c_lo);
  return S;
}

// The gradient's factors: d_v = A 2^((s_v - all.ref) c) - p_v for a token of the list, less
// B 2^((s_v - rest.ref) c) for any other; C covers both terms of the latter with one exponential
// unless the two references lie too far apart for fp32 (one false).
struct Factors {
  float A, B, C;
  bool one;
  __device__ __forceinline__ Factors(float scale, float er, float invE, const Sum2& all, const Sum2& rest, float c) {
    A = all.s > 0.0f && all.s < INFINITY ? scale / all.s : NAN;
    B = er != 0.0f ? scale * (er * invE) / rest.s : 0.0f;
    const float apart = (all.ref - rest.ref) * c;
    one = er == 0.0f || apart < 80.0f;
    C = er == 0.0f ? A : A - B * ex2(apart);
  }
  __device__ __forceinline__ float outside(float s, const Sum2& all, const Sum2& rest, float c) const {
    const float a = ex2((s - all.ref) * c);
    return one ? C * a : A * a - B * ex2((s - rest.ref) * c);
  }
};
// From the list's masses, against ref, to the whole row's reference (a list of -inf has none, and a
// reference that may lie far above the row).
__device__ __forceinline__ float list_factor(const F2& list, float ref, const Sum2& all, float c) {
  return list.value() == 0.0f ? 0.0f : ex2((ref - all.ref) * c);
}
template <bool kBF16>
__device__ __forceinline__ void put_grad(unsigned char* base, int v, float d) {
  if (kBF16) reinterpret_cast<__nv_bfloat16*>(base)[v] = __float2bfloat16_rn(d);
  else reinterpret_cast<float*>(base)[v] = d;
}
// The gradient of a vector's tokens: C 2^(x c - rc).
template <bool kBF16>
__device__ __forceinline__ uint4 grad_vec(const uint4& w, f32x2 c2, f32x2 nrc2, f32x2 C2) {
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < (kBF16 ? 4 : 2); ++i) {
    float a, b;
    unpack2(fma2(pair_of<kBF16>(w, i), c2, nrc2), a, b);
    unpack2(mul2(pack2(ex2(a), ex2(b)), C2), a, b);
    if (kBF16) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);  // the gradient's one rounding
      out[i] = reinterpret_cast<const uint32_t&>(h);
    } else {
      out[2 * i] = __float_as_uint(a);
      out[2 * i + 1] = __float_as_uint(b);
    }
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}
// The gradient of the list's tokens, over what is there: at element id of place(id) (nullptr:
// another CTA's).  A token of several slots (dup: there are some) takes the sum of their masses in
// slot order, at its first slot.  s_e, s_v: the teacher's and the student's masses before their
// factors unit and A.
template <bool kBF16, class Place>
__device__ __forceinline__ void put_listed(Place&& place, bool dup, int K, const int32_t* s_id, const float* s_e,
                                           const float* s_v, float A, float unit) {
  for (int k = threadIdx.x; k < K; k += kNT) {
    const int32_t id = s_id[k];
    unsigned char* base = id >= 0 ? place(id) : nullptr;  // empty slots are -1
    if (!base) continue;
    float e = s_e[k];
    if (dup) {
      e = 0.0f;
      bool first = true;
      for (int j = 0; j < K; ++j) {
        if (s_id[j] != id) continue;
        first = first && j >= k;
        e += s_e[j];
      }
      if (!first) continue;
    }
    put_grad<kBF16>(base, id, A * s_v[k] - unit * e);
  }
}

// The list's tokens among the elements of a CTA's i-th vector (its bitmap starts one vector early).
template <bool kBF16>
__device__ __forceinline__ uint32_t listed_bits(const unsigned char* bytes, int i, bool in) {
  const int b = (i + 1) * (kBF16 ? 8 : 4);
  const uint32_t m = in ? bytes[b >> 3] : 0u;
  return kBF16 ? m : (m >> (b & 4)) & 15u;
}
// The thread's sum over vectors [g0, g1) of a row, without the list's tokens, and one logit more,
// with a reference that moves up: for rows whose list lies far from everything else.
template <bool kBF16>
__device__ __noinline__ Sum2 moving_sum(const RowView<kBF16>& x, int g0, int g1, const unsigned char* bytes, float one, float c) {
  Sum2 sum{-FLT_MAX, 0.0f};
  for (int g = g0 + static_cast<int>(threadIdx.x); g < g1; g += kNT) {
    uint4 v = ld_stream(x.vec + g);
    drop_listed<kBF16>(v, listed_bits<kBF16>(bytes, g - g0, true));
    const float m = vec_max<kBF16>(v);
    if ((m - sum.ref) * c > kRaise) sum.raise(clamp_ref(m), c);
    add_vec<kBF16>(sum, v, c);
  }
  add_one(sum, one, c);
  return sum;
}

// kRest (backward): whether the teacher has a rest; the loss's modes always split the row's sum (launch).
template <bool kBF16, int kMode, bool kRest = true>
__global__ void __launch_bounds__(kNT, Flight<kMode>::ctas) distill_kernel(const Params P) {
  constexpr int G = kBF16 ? 8 : 4, kU = Flight<kMode>::loads;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float red[kNW][2];
  __shared__ float part[kMaxCS][2];  // the partial sums of the cluster's CTAs
  __shared__ F2 sums[kNW][3];        // per warp: E, W and the student's sum over the list
  __shared__ uint32_t top[2];
  __shared__ int flags[2];
  static_assert(kRest || kMode == kBackward);
  const int CS = static_cast<int>(cg::this_cluster().num_blocks());
  const int rank = static_cast<int>(cg::this_cluster().block_rank());
  const int64_t row = blockIdx.x / CS;
  // every CTA of the cluster runs before any writes into another's shared memory
  constexpr bool kShare = kMode != kBackward;  // the cluster's CTAs exchange their partial sums
  if (kShare && CS > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  const int V = P.V, K = P.K;
  const float c = P.c;

  const RowView<kBF16> x(P.student, row * P.ld, V);
  const int g0 = static_cast<int>(static_cast<int64_t>(x.nv) * rank / CS);
  const int g1 = static_cast<int>(static_cast<int64_t>(x.nv) * (rank + 1) / CS);
  const Layout lay = make_layout(K, (V + CS - 1) / CS + 4 * G, kMode != kBackward);
  int32_t* s_id = reinterpret_cast<int32_t*>(smem + lay.id);
  float* s_e = reinterpret_cast<float*>(smem + lay.e);
  float* s_v = reinterpret_cast<float*>(smem + lay.v);
  int32_t* s_hash = reinterpret_cast<int32_t*>(smem + lay.hash);
  uint32_t* s_bits = reinterpret_cast<uint32_t*>(smem + lay.bits);
  // bit of element v: its distance from the first element of vector g0, plus G (the head's
  // elements come before the first vector)
  const int bit0 = x.head + g0 * G - G;
  const int nbits = (g1 - g0 + 3) * G;

  // ---- the teacher's slots ------------------------------------------------------------
  if (threadIdx.x < 2) {
    top[threadIdx.x] = 0u;
    flags[threadIdx.x] = 0;
  }
  if (kMode != kBackward)
    for (int i = threadIdx.x; i < (nbits + 31) / 32; i += kNT) s_bits[i] = 0u;
  for (int i = threadIdx.x; i < lay.hash_size; i += kNT) s_hash[i] = -1;
  // (the slots of a row of weight 0 are read all the same: their loads need not wait for the weight's)
  Slot slot = first_slot(P, row);
  const float w = P.weight ? P.weight[row] : 1.0f;
  const float r = kRest && P.rest ? P.rest[row] : -INFINITY;
  float scale = w;  // of the gradient
  if (kMode != kForward && P.upstream) scale *= P.upstream[row];
  scale *= P.tau;
  __syncthreads();
  if (w != 0.0f)
    read_slots(P, row, x, slot, s_id, s_e, s_v, s_hash, lay.hash_size, top, flags, [&](int, int32_t id) {
      const int b = id - bit0;
      if (kMode != kBackward && b >= 0 && b < nbits) atomicOr(&s_bits[b >> 5], 1u << (b & 31));
    });
  __syncthreads();
  if (kShare && CS > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (!flags[0] || (kMode == kBackward && scale == 0.0f)) {
    // no loss: zeros, and the student's row is not looked at (the same in every CTA of the row)
    if (rank == 0 && threadIdx.x == 0) {
      if (kMode != kBackward) P.loss[row] = 0.0f;
      if (kMode == kForward && P.stats)
        for (int i = 0; i < kStats; ++i) P.stats[row * kStats + i] = 0.0f;
    }
    if (kMode != kForward) zero_row<kBF16>(P.grad, row * P.ld_grad, V, rank, CS);
    return;
  }
  const bool dup = flags[1] != 0;
  // the student's sums: over the whole row, and over the tokens outside the list
  Sum2 all, rest;
  if (kMode == kBackward) {
    all = Sum2{P.stats[row * kStats], P.stats[row * kStats + 1]};
    rest = Sum2{P.stats[row * kStats + 2], P.stats[row * kStats + 3]};
  }
  const float tref = teacher_ref(top, r, P.tau);
  const float ref = kMode == kBackward ? all.ref : student_ref(top);
  slot_masses(P, K, tref, ref, dup, s_id, s_e, s_v, sums);  // read after the barriers below

  // ---- the student's sum outside the list --------------------------------------------------------
  // Against the list's largest logit, one reference for the whole row and near its top.  A sum that
  // leaves fp32's range (the list far from everything else) is taken again with moving references.
  if (kMode != kBackward) {
    const unsigned char* bytes = reinterpret_cast<const unsigned char*>(s_bits);
    // the element outside the vectors that is this thread's, if any: the head's with rank 0, the
    // tail's with the last rank
    const bool loose = static_cast<int>(threadIdx.x) < x.loose() &&
                       ((x.loose_at(threadIdx.x) < x.head) ? rank == 0 : rank == CS - 1);
    const int lv = loose ? x.loose_at(threadIdx.x) : 0;
    const bool loose_out = loose && !((s_bits[(lv - bit0) >> 5] >> ((lv - bit0) & 31)) & 1u);
    FastSum<kBF16> fast(fabsf(ref * c) <= kFastRef ? ref : 0.0f, c);
    for (int base = g0; base < g1; base += kNT * kU) {
      uint4 v[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int g = base + u * kNT + static_cast<int>(threadIdx.x);
        v[u] = g < g1 ? ld_stream(x.vec + g) : neg_inf_vec<kBF16>();
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int g = base + u * kNT + static_cast<int>(threadIdx.x);
        const uint32_t m = listed_bits<kBF16>(bytes, g - g0, g < g1);
        if (m) drop_listed<kBF16>(v[u], m);
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) fast.add(v[u]);
    }
    rest = Sum2{ref, fast.total(ref, c)};
    // (against the one reference too: a sum of its own would hide, in the merge, that others overflow)
    if (loose_out) rest.s += ex2((x.at(lv) - ref) * c);
    Teacher T;
    F2 S;
    Sum2 list;
    for (bool moving = false;; moving = true) {
      if (moving) rest = moving_sum<kBF16>(x, g0, g1, bytes, loose_out ? x.at(lv) : -INFINITY, c);
      rest = block_merge(rest, c, red);
      if (!moving) {
        S = collect<true>(sums, K, r, tref, P.tau, c, P.c_lo, T);
        list = Sum2{ref, S.value()};
      }
      if (CS > 1) {
        cg::cluster_group cl = cg::this_cluster();
        if (static_cast<int>(threadIdx.x) < CS) {
          float* to = cl.map_shared_rank(&part[0][0], threadIdx.x);
          to[2 * rank] = rest.ref;
          to[2 * rank + 1] = rest.s;
        }
        cl.sync();  // every CTA holds every part
        rest = Sum2{part[0][0], part[0][1]};
        for (int q = 1; q < CS; ++q) rest = merge(rest, Sum2{part[q][0], part[q][1]}, c);
      }
      all = merge(list, rest, c);
      // the same in every CTA
      if (moving || (fabsf(ref * c) <= kFastRef && precise(rest, list, T.er) && all.s <= 0x1p100f)) break;
      if (CS > 1) cg::this_cluster().sync();  // the parts are read
    }
    if (rank == 0 && threadIdx.x == 0) {
      P.loss[row] = row_loss(P, T, ref, S, rest, all, w);
      if (kMode == kForward && P.stats) {
        P.stats[row * kStats] = all.ref;
        P.stats[row * kStats + 1] = all.s;
        P.stats[row * kStats + 2] = rest.ref;
        P.stats[row * kStats + 3] = rest.s;
      }
    }
    if (kMode == kForward) return;
  } else {
    __syncthreads();  // the slots' masses
  }

  // ---- the gradient -------------------------------------------------------------------
  if (kMode != kForward) {
    Teacher T;
    const F2 S = collect<kRest>(sums, K, r, tref, P.tau, c, P.c_lo, T);
    const float invE = 1.0f / (T.E.value() + T.er);
    const Factors F(scale, T.er, invE, all, rest, c);
    const RowView<kBF16> o(P.grad, row * P.ld_grad, V);
    unsigned char* obase = const_cast<unsigned char*>(o.base);
    const float rc = all.ref * c;
    if (F.one && o.head == x.head && fabsf(rc) <= kFastRef) {
      const float fix = ex2(-fmaf(all.ref, c, -rc));  // what rc's rounding left out
      const f32x2 nrc2 = pack2(-rc, -rc), c2 = pack2(c, c), C2 = pack2(F.C * fix, F.C * fix);
      uint4* ov = const_cast<uint4*>(o.vec);
      for (int base = g0; base < g1; base += kNT * kU) {
        uint4 v[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int g = base + u * kNT + static_cast<int>(threadIdx.x);
          v[u] = g < g1 ? ld_stream(x.vec + g) : neg_inf_vec<kBF16>();
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int g = base + u * kNT + static_cast<int>(threadIdx.x);
          if (g < g1) __stcs(ov + g, grad_vec<kBF16>(v[u], c2, nrc2, C2));
        }
      }
      if (static_cast<int>(threadIdx.x) < x.loose()) {
        const int v = x.loose_at(threadIdx.x);
        if ((v < x.head) ? rank == 0 : rank == CS - 1) put_grad<kBF16>(obase, v, F.outside(x.at(v), all, rest, c));
      }
    } else {
      // the two rows do not share their 16-byte boundaries, or the numbers are extreme: one
      // element at a time
      const int v0 = rank == 0 ? 0 : x.head + g0 * G;
      const int v1 = rank == CS - 1 ? V : x.head + g1 * G;
      for (int v = v0 + static_cast<int>(threadIdx.x); v < v1; v += kNT)
        put_grad<kBF16>(obase, v, F.outside(x.at(v), all, rest, c));
    }
    // the list's tokens in this CTA's part, over what the pass above wrote
    __syncthreads();
    const int v0 = rank == 0 ? 0 : x.head + g0 * G, v1 = rank == CS - 1 ? V : x.head + g1 * G;
    put_listed<kBF16>([&](int32_t id) { return id >= v0 && id < v1 ? obase : nullptr; }, dup, K, s_id, s_e, s_v,
                      F.A * list_factor(S, ref, all, c), scale * invE);
  }
}

// ------------------------------------------------------------------------------------------
// The loss and the gradient with the row in shared memory
// ------------------------------------------------------------------------------------------
//
// Memory bounds the pair: the row is read once, by a bulk copy into the shared memory of each of a
// cluster's CTAs, summed there, turned into the gradient in place and copied out.  Read again from
// global memory instead it came from DRAM once more (an SM's rows in flight, times 152, are more
// than the second-level cache holds): 495 us for 4096 rows of 151936 bf16 with a quarter masked
// (321 us at the copy rate), whatever the number of rows in flight.  What it took since: copies by
// the threads 437 us, bulk copies 409, the cluster's sums sent with stores that count at their
// receiver's barrier instead of a cluster barrier (whose fence waits for everything) 395, a first
// cluster barrier without a fence 368, and four CTAs' registers 363 (five CTAs': 370; shared memory
// holds four).  1024 rows of 128256: 91 us (77 at the copy rate).  What bounds it now is the time
// that a part of a row spends waiting between its slots' loads and its last byte out: memory is
// busy for 88% of it.
//
// Bytes of a row per CTA, where the cluster allows: four CTAs an SM.  40 KB took 386 us, 44 KB 408,
// 62 KB 403 (fewer CTAs to fill each other's waits).
constexpr int kChunkBytes = 52 * 1024;

// What the host lays out for a launch: `share` vectors of a row for each CTA, and the offsets of
// the small arrays behind them in shared memory.
struct Resident {
  int share, hash_size;
  int id, e, v, next, head, hash;
};

template <bool kBF16>
__global__ void __launch_bounds__(kNT, 4) distill_resident_kernel(const Params P, const Resident R) {
  constexpr int G = kBF16 ? 8 : 4;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float part[kMaxCS * kNW];  // per warp of the cluster
  __shared__ F2 teacher[kNW][3];        // per warp: E, W and the student's sum over the list
  __shared__ uint32_t top[2];           // keys of the largest teacher's value and student's logit in the list
  __shared__ int flags[2];              // the row has a filled slot; some token has two
  __shared__ __align__(8) unsigned long long landed, gathered;  // the barriers of the copy and of part[]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  cg::cluster_group cl = cg::this_cluster();
  const int CS = static_cast<int>(cl.num_blocks());
  const int rank = static_cast<int>(cl.block_rank());
  uint32_t cluster;
  asm("mov.u32 %0, %%clusterid.x;" : "=r"(cluster));
  const int64_t row = cluster;
  const int V = P.V, K = P.K;
  const float c = P.c;
  if (threadIdx.x == 0) {
    copy_barrier_init(&landed);
    copy_barrier_init(&gathered);
    if (CS > 1) expect_bytes(&gathered, static_cast<uint32_t>(kNW * CS * sizeof(float)));
  }
  __syncwarp();
  // every CTA of the cluster runs, and has set up its barriers, before any writes into another's
  // shared memory.  The barriers' own fence is behind their setting up; an arrival that releases
  // would fence for every thread (394 us against 368).
  if (CS > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const RowView<kBF16> x(P.student, row * P.ld, V);
  const int g0 = min(rank * R.share, x.nv), g1 = rank == CS - 1 ? x.nv : min(g0 + R.share, x.nv);
  const int g = g0 + static_cast<int>(threadIdx.x);                  // the thread's vectors: g + i kNT, i < count,
  uint4* const mine = reinterpret_cast<uint4*>(smem) + threadIdx.x;  // kept at mine[i kNT]
  const int count = g < g1 ? (g1 - g - 1) / kNT + 1 : 0;
  int32_t* s_id = reinterpret_cast<int32_t*>(smem + R.id);
  float* s_e = reinterpret_cast<float*>(smem + R.e);
  float* s_v = reinterpret_cast<float*>(smem + R.v);
  int32_t* s_next = reinterpret_cast<int32_t*>(smem + R.next);
  int32_t* s_head = reinterpret_cast<int32_t*>(smem + R.head);  // per thread: the first of the slots whose tokens
  int32_t* s_hash = reinterpret_cast<int32_t*>(smem + R.hash);  // lie in its vectors, the others by s_next

  // ---- the copy, and the teacher's slots while it is under way ------------------------------------
  if (threadIdx.x < 2) {
    top[threadIdx.x] = 0u;
    flags[threadIdx.x] = 0;
  }
  s_head[threadIdx.x] = -1;
  for (int i = threadIdx.x; i < R.hash_size; i += kNT) s_hash[i] = -1;
  // (the slots of a row of weight 0 are read all the same: their loads need not wait for the weight's)
  Slot slot = first_slot(P, row);
  const float w = P.weight ? P.weight[row] : 1.0f;
  const float r = P.rest ? P.rest[row] : -INFINITY;
  const float scale = w * P.tau;
  __syncthreads();
  if (w != 0.0f) {
    if (threadIdx.x == 0 && g1 > g0) copy_in(smem, x.vec + g0, static_cast<uint32_t>(g1 - g0) * 16u, &landed);
    read_slots(P, row, x, slot, s_id, s_e, s_v, s_hash, R.hash_size, top, flags, [&](int k, int32_t id) {
      const int at = id - x.head, vec = at / G - g0;
      if (at >= 0 && vec >= 0 && vec < g1 - g0) s_next[k] = atomicExch(&s_head[vec & (kNT - 1)], k);
    });
  }
  __syncthreads();
  if (!flags[0]) {  // no loss: zeros (the same in every CTA of the row)
    if (w != 0.0f && g1 > g0) copy_landed(&landed);
    if (CS > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (rank == 0 && threadIdx.x == 0) P.loss[row] = 0.0f;
    zero_row<kBF16>(P.grad, row * P.ld_grad, V, rank, CS);
    return;
  }
  const bool dup = flags[1] != 0;
  const float tref = teacher_ref(top, r, P.tau), ref = student_ref(top);  // the latter of the student's sums too
  slot_masses(P, K, tref, ref, dup, s_id, s_e, s_v, teacher);

  // ---- the student's sum outside the list -------------------------------------------------------
  // The list's tokens leave the row: each thread overwrites those in its own vectors with
  // -inf (their logits are in s_v).  Against the list's largest student logit, one reference for
  // the whole row, so that the parts simply add up; a sum that leaves fp32's range (the list far
  // from everything else) is taken again below against its own maximum.
  bool late = g1 > g0 && !copy_landed(&landed);  // a wait ran out
  float s_rest;
  {
    FastSum<kBF16> fast(fabsf(ref * c) <= kFastRef ? ref : 0.0f, c);
    for (int k = s_head[threadIdx.x]; k >= 0; k = s_next[k]) {
      const int at = s_id[k] - x.head;
      uint4* v = mine + (at / G - g);
      if (kBF16) reinterpret_cast<uint16_t*>(v)[at % G] = 0xFF80u;
      else reinterpret_cast<uint32_t*>(v)[at % G] = 0xFF800000u;
    }
#pragma unroll 4
    for (int i = 0; i < count; ++i) fast.add(mine[i * kNT]);
    s_rest = late ? NAN : fast.total(ref, c);  // a row that did not arrive has no result
  }
  // the elements outside the vectors: the head with rank 0, the tail with the last rank
  const bool has_loose = static_cast<int>(threadIdx.x) < x.loose() &&
                         ((x.loose_at(threadIdx.x) < x.head) ? rank == 0 : rank == CS - 1);
  const int loose_v = has_loose ? x.loose_at(threadIdx.x) : 0;
  const float loose_s = has_loose ? x.at(loose_v) : -INFINITY;
  const bool loose_out = has_loose && !has_token(s_hash, R.hash_size, loose_v);
  if (loose_out) s_rest += ex2((loose_s - ref) * c);
  if (CS > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // (of the arrival at the top)
  // Gives every warp of the cluster's CTAs' values a to all of them, at part[].
  auto exchange = [&](float a) {
    if (CS > 1) {
      if (lane < CS) *cl.map_shared_rank(&part[rank * kNW + warp], lane) = a;
      cl.sync();
    } else {
      if (lane == 0) part[warp] = a;
      __syncthreads();
    }
  };
  auto part_sum = [&]() -> float {
    float t = lane < kNW * CS ? part[lane] : 0.0f;
    if (lane + 32 < kNW * CS) t += part[lane + 32];
    return warp_sum(t);
  };
  {
    // the same with stores that count at the receiver's barrier: no fence, and no CTA waits for
    // more than the values
    const float a = warp_sum(s_rest);
    if (CS > 1) {
      if (lane < CS) send_float(&part[rank * kNW + warp], a, &gathered, lane);
      if (!copy_landed(&gathered)) late = true;
    } else if (lane == 0) {
      part[warp] = a;
    }
    __syncthreads();  // (the slots' sums, too)
  }
  Teacher T;
  const F2 S = collect<true>(teacher, K, r, tref, P.tau, c, P.c_lo, T);
  const Sum2 list{ref, S.value()};
  Sum2 rest{ref, late ? NAN : part_sum()};
  Sum2 all{ref, rest.s + list.s};
  // (NaN fails this too)
  if (!(fabsf(ref * c) <= kFastRef && precise(rest, list, T.er) && all.s <= 0x1p100f)) {
    // the same in every CTA: the largest logit outside the list (NaN: there is one), then the sum
    // against that
    float m = loose_out ? loose_s : -INFINITY;
    bool nan = late || isnan(m);
    auto each = [&](auto&& f) {
      for (int i = 0; i < count; ++i) {
        const uint4 v = mine[i * kNT];
        const uint32_t word[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < G; ++e)
          f(kBF16 ? __uint_as_float((e & 1) ? (word[e / 2] & 0xFFFF0000u) : (word[e / 2] << 16)) : __uint_as_float(word[e]));
      }
    };
    each([&](float y) {
      m = fmaxf(m, y);
      nan |= isnan(y);
    });
    nan = __any_sync(0xffffffffu, nan);
    m = nan ? NAN : warp_max(m);
    if (CS > 1) cl.sync(); else __syncthreads();  // the parts are read
    exchange(m);
    m = -INFINITY;
    nan = false;
    for (int i = 0; i < kNW * CS; ++i) {
      m = fmaxf(m, part[i]);
      nan |= isnan(part[i]);
    }
    m = clamp_ref(m);
    float t = loose_out ? ex2((loose_s - m) * c) : 0.0f;
    each([&](float y) { t += ex2((y - m) * c); });
    if (CS > 1) cl.sync(); else __syncthreads();
    exchange(warp_sum(t));
    rest = Sum2{m, part_sum()};
    all = merge(list, rest, c);
    if (nan) all.s = NAN;
  }
  // ---- the gradient ------------------------------------------------------------------------------
  // In place in shared memory, the list's tokens last, and out with one copy.
  const float invE = 1.0f / (T.E.value() + T.er);
  const Factors F(scale, T.er, invE, all, rest, c);
  const RowView<kBF16> o(P.grad, row * P.ld_grad, V);
  unsigned char* obase = const_cast<unsigned char*>(o.base);
  unsigned char* inside = obase;  // where element id of this CTA's vectors goes
  const int v0 = x.head + g0 * G, v1 = x.head + g1 * G;
  const float rc = all.ref * c;
  if (F.one && o.head == x.head && fabsf(rc) <= kFastRef) {
    const float fix = ex2(-fmaf(all.ref, c, -rc));  // what rc's rounding left out
    const f32x2 nrc2 = pack2(-rc, -rc), c2 = pack2(c, c), C2 = pack2(F.C * fix, F.C * fix);
#pragma unroll 4
    for (int i = 0; i < count; ++i) mine[i * kNT] = grad_vec<kBF16>(mine[i * kNT], c2, nrc2, C2);
    inside = smem - static_cast<int64_t>(v0) * (kBF16 ? 2 : 4);
  } else {
    for (int i = 0; i < count; ++i) {
      const uint4 v = mine[i * kNT];
      const uint32_t word[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < G; ++e) {
        const float s = kBF16 ? __uint_as_float((e & 1) ? (word[e / 2] & 0xFFFF0000u) : (word[e / 2] << 16))
                              : __uint_as_float(word[e]);
        put_grad<kBF16>(obase, v0 + (static_cast<int>(threadIdx.x) + i * kNT) * G + e, F.outside(s, all, rest, c));
      }
    }
  }
  if (has_loose) put_grad<kBF16>(obase, loose_v, F.outside(loose_s, all, rest, c));
  __syncthreads();
  put_listed<kBF16>(
      [&](int32_t id) -> unsigned char* {
        if (id >= v0 && id < v1) return inside;
        return (rank == 0 && id < x.head) || (rank == CS - 1 && id >= v1) ? obase : nullptr;
      },
      dup, K, s_id, s_e, s_v, F.A * list_factor(S, ref, all, c), scale * invE);
  if (inside != obase) {
    publish_to_copies();
    __syncthreads();
    if (threadIdx.x == 0 && g1 > g0)
      copy_out(const_cast<uint4*>(o.vec) + g0, smem, static_cast<uint32_t>(g1 - g0) * 16u);
  }
  if (rank == 0 && threadIdx.x == kNT - 1) P.loss[row] = row_loss(P, T, ref, S, rest, all, w);
  if (late) copy_landed(&landed);  // one more wait before the block leaves
}

// ------------------------------------------------------------------------------------------
// Host side
// ------------------------------------------------------------------------------------------
static int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    (void)cudaGetLastError();
    return 0;
  }
  return n;
}

// Lets a kernel take as much dynamic shared memory as a block can have: the same for every call,
// so that calls side by side do not undo each other's; once for each device.
constexpr int kMaxDynamic = 224 * 1024;
template <class Kernel>
static bool allow_shared(Kernel* kernel, std::atomic<bool>* done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
  if (done[dev].load(std::memory_order_acquire)) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxDynamic) != cudaSuccess) return false;
  done[dev].store(true, std::memory_order_release);
  return true;
}

template <bool kBF16, int kMode, bool kRest = true>
static kps_status launch_t(const Params& P, cudaStream_t stream) {
  const int sms = sm_count();
  if (!sms) return KPS_ERR_CUDA;
  // few rows: a cluster shares each, as wide as leaves every thread four vectors
  int cs = 1;
  const int64_t round = static_cast<int64_t>(kNT) * 4 * (kBF16 ? 8 : 4);
  while (cs < kMaxCS && P.N * cs * 2 <= 2 * sms && P.V >= 2 * cs * round) cs *= 2;
  const Layout lay = make_layout(P.K, (P.V + cs - 1) / cs + 4 * (kBF16 ? 8 : 4), kMode != kBackward);
  static std::atomic<bool> done[kMaxDevices];
  if (!allow_shared(distill_kernel<kBF16, kMode, kRest>, done)) {
    (void)cudaGetLastError();
    return KPS_ERR_CUDA;
  }
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(static_cast<unsigned>(P.N * cs));
  lc.blockDim = dim3(kNT);
  lc.dynamicSmemBytes = lay.total;
  lc.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  if (cudaLaunchKernelEx(&lc, distill_kernel<kBF16, kMode, kRest>, P) != cudaSuccess) {
    (void)cudaGetLastError();
    return KPS_ERR_CUDA;
  }
  return KPS_OK;
}

// The loss and the gradient: with the row in shared memory where a cluster's holds it.
template <bool kBF16>
static kps_status launch_both(const Params& P, cudaStream_t stream) {
  const int sms = sm_count();
  if (!sms) return KPS_ERR_CUDA;
  constexpr int G = kBF16 ? 8 : 4;
  const int64_t bytes = static_cast<int64_t>(P.V) * (kBF16 ? 2 : 4);
  int cs = static_cast<int>((bytes + kChunkBytes - 1) / kChunkBytes);
  cs = cs < 1 ? 1 : cs > kMaxCS ? kMaxCS : cs;
  // few rows: wider clusters, while every thread keeps a group's worth of vectors
  while (2 * cs <= kMaxCS && P.N * cs * 2 <= 2 * sms && P.V >= 2 * cs * kNT * 4 * G) cs *= 2;
  Resident R;
  R.share = (P.V / G + cs - 1) / cs;
  R.hash_size = 32;
  while (R.hash_size < 2 * P.K) R.hash_size *= 2;
  const int k4 = (P.K * 4 + 15) / 16 * 16;
  R.id = (R.share + kNT - 1) / kNT * kNT * 16;  // a whole round of vectors for every thread
  R.e = R.id + k4;
  R.v = R.e + k4;
  R.next = R.v + k4;
  R.head = R.next + k4;
  R.hash = R.head + kNT * 4;
  const size_t total = static_cast<size_t>(R.hash) + R.hash_size * 4;
  // a row's part and the list's arrays have to fit together
  if (total > kMaxDynamic) return launch_t<kBF16, kBoth>(P, stream);
  auto* kernel = distill_resident_kernel<kBF16>;
  static std::atomic<bool> done[kMaxDevices];
  if (!allow_shared(kernel, done)) {
    (void)cudaGetLastError();
    return KPS_ERR_CUDA;
  }
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(static_cast<unsigned>(P.N * cs));
  lc.blockDim = dim3(kNT);
  lc.dynamicSmemBytes = total;
  lc.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  if (cudaLaunchKernelEx(&lc, kernel, P, R) != cudaSuccess) {
    (void)cudaGetLastError();
    return KPS_ERR_CUDA;
  }
  return KPS_OK;
}

template <int kMode>
static kps_status launch(const Params& P, kps_dtype dt, cudaStream_t stream) {
  // The loss always takes the list's tokens out of the row's sum, rest or not: they weigh most where
  // the student is near its teacher, and the loss, a small number there, then comes from sums in two
  // floats (without a rest its error against 64 bits fell from 1e-6 to 1.2e-7; 1024 rows of 128256
  // bf16 take 49 us instead of 44).
  if (kMode == kBoth) return dt == KPS_BF16 ? launch_both<true>(P, stream) : launch_both<false>(P, stream);
  if (kMode == kForward || P.rest)
    return dt == KPS_BF16 ? launch_t<true, kMode>(P, stream) : launch_t<false, kMode>(P, stream);
  return dt == KPS_BF16 ? launch_t<true, kBackward, false>(P, stream) : launch_t<false, kBackward, false>(P, stream);
}

// The checks every entry point shares; fills P.  *empty: nothing to do.
static kps_status check(const void* student, kps_dtype dt, int64_t N, int64_t V, int64_t ld, const int32_t* ids,
                        const void* values, kps_dtype values_dt, int64_t K, const float* rest, const float* weight,
                        float temperature, Params* P) {
  if ((dt != KPS_F32 && dt != KPS_BF16) || (values_dt != KPS_F32 && values_dt != KPS_BF16)) return KPS_ERR_INVALID_ARG;
  if (N < 0 || V < 1 || K < 1 || K > kMaxK) return KPS_ERR_INVALID_ARG;
  if (N > 1 && ld < V) return KPS_ERR_INVALID_ARG;
  // the loss holds the temperature's square, which has to be a normal number
  const float tau2 = temperature * temperature;
  if (!(temperature > 0.0f) || !(tau2 >= FLT_MIN) || std::isinf(tau2)) return KPS_ERR_INVALID_ARG;
  if (V > kMaxV || N > INT32_MAX / kMaxCS) return KPS_ERR_UNSUPPORTED;
  if (N == 0) return KPS_OK;
  if (!student || !ids || !values) return KPS_ERR_INVALID_ARG;
  const uintptr_t esize = dt == KPS_BF16 ? 2 : 4, vsize = values_dt == KPS_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(student) % esize || reinterpret_cast<uintptr_t>(values) % vsize ||
      reinterpret_cast<uintptr_t>(ids) % 4 || reinterpret_cast<uintptr_t>(rest) % 4 || reinterpret_cast<uintptr_t>(weight) % 4)
    return KPS_ERR_INVALID_ARG;
  P->student = student;
  P->N = N;
  P->ld = ld;
  P->V = static_cast<int>(V);
  P->K = static_cast<int>(K);
  P->ids = ids;
  P->values = values;
  P->values_bf16 = values_dt == KPS_BF16;
  P->rest = rest;
  P->weight = weight;
  P->tau = temperature;
  const double c = 1.4426950408889634074 / static_cast<double>(temperature);
  P->c = static_cast<float>(c);
  P->c_lo = static_cast<float>(c - static_cast<double>(P->c));
  return KPS_OK;
}

static bool float_aligned(const void* p) { return reinterpret_cast<uintptr_t>(p) % alignof(float) == 0; }

// A gradient buffer of its own: rows of at least V elements, sharing no byte with the student's rows.
static kps_status check_grad(const Params& P, kps_dtype dt, void* grad, int64_t ld_grad) {
  const uintptr_t esize = dt == KPS_BF16 ? 2 : 4;
  if (!grad || reinterpret_cast<uintptr_t>(grad) % esize || (P.N > 1 && ld_grad < P.V)) return KPS_ERR_INVALID_ARG;
  const uintptr_t a = reinterpret_cast<uintptr_t>(P.student), b = reinterpret_cast<uintptr_t>(grad);
  const uintptr_t an = ((P.N - 1) * P.ld + P.V) * esize, bn = ((P.N - 1) * ld_grad + P.V) * esize;
  if (a < b + bn && b < a + an) return KPS_ERR_INVALID_ARG;
  return KPS_OK;
}

}  // namespace distill
}  // namespace kps

extern "C" {

kps_status kps_distill_forward(const void* student, kps_dtype dt, int64_t N, int64_t V, int64_t ld,
                               const int32_t* ids, const void* values, kps_dtype values_dt, int64_t K,
                               const float* rest, const float* weight, float temperature, float* out_loss,
                               float* out_stats, cudaStream_t stream) {
  const kps::NvtxRange range("kps_distill_forward");
  kps::distill::Params P = {};
  const kps_status st = kps::distill::check(student, dt, N, V, ld, ids, values, values_dt, K, rest, weight, temperature, &P);
  if (st != KPS_OK || N == 0) return st;
  if (!out_loss || !kps::distill::float_aligned(out_loss) || !kps::distill::float_aligned(out_stats)) return KPS_ERR_INVALID_ARG;
  P.loss = out_loss;
  P.stats = out_stats;
  return kps::distill::launch<kps::distill::kForward>(P, dt, stream);
}

kps_status kps_distill_backward(const void* student, kps_dtype dt, int64_t N, int64_t V, int64_t ld,
                                const int32_t* ids, const void* values, kps_dtype values_dt, int64_t K,
                                const float* rest, const float* weight, float temperature, const float* grad_loss,
                                const float* stats, void* out_grad, int64_t ld_grad, cudaStream_t stream) {
  const kps::NvtxRange range("kps_distill_backward");
  kps::distill::Params P = {};
  kps_status st = kps::distill::check(student, dt, N, V, ld, ids, values, values_dt, K, rest, weight, temperature, &P);
  if (st != KPS_OK || N == 0) return st;
  if (!stats || !kps::distill::float_aligned(stats) || !kps::distill::float_aligned(grad_loss)) return KPS_ERR_INVALID_ARG;
  if ((st = kps::distill::check_grad(P, dt, out_grad, ld_grad)) != KPS_OK) return st;
  P.upstream = grad_loss;
  P.stats = const_cast<float*>(stats);
  P.grad = out_grad;
  P.ld_grad = ld_grad;
  return kps::distill::launch<kps::distill::kBackward>(P, dt, stream);
}

kps_status kps_distill_loss_grad(const void* student, kps_dtype dt, int64_t N, int64_t V, int64_t ld,
                                 const int32_t* ids, const void* values, kps_dtype values_dt, int64_t K,
                                 const float* rest, const float* weight, float temperature, float* out_loss,
                                 void* out_grad, int64_t ld_grad, cudaStream_t stream) {
  const kps::NvtxRange range("kps_distill_loss_grad");
  kps::distill::Params P = {};
  kps_status st = kps::distill::check(student, dt, N, V, ld, ids, values, values_dt, K, rest, weight, temperature, &P);
  if (st != KPS_OK || N == 0) return st;
  if (!out_loss || !kps::distill::float_aligned(out_loss)) return KPS_ERR_INVALID_ARG;
  if ((st = kps::distill::check_grad(P, dt, out_grad, ld_grad)) != KPS_OK) return st;
  P.loss = out_loss;
  P.grad = out_grad;
  P.ld_grad = ld_grad;
  return kps::distill::launch<kps::distill::kBoth>(P, dt, stream);
}

}  // extern "C"
