// kps_stream.cuh — streaming one row of logits through a thread block: the row's 16-byte
// vectors, packed fp32 arithmetic, base-2 sums of exponentials and their reductions.  Shared
// by the kernels that read whole rows of [rows, vocab] logits (the top logits, distillation).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cfloat>
#include <cstdint>

namespace kps {
namespace stream {

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;
// The vectors of one row: `head` elements before the first 16-byte boundary, `nv` vectors of G
// elements, then the tail.
template <bool kBF16>
struct RowView {
  static constexpr int G = kBF16 ? 8 : 4;
  const unsigned char* base;  // element 0
  const uint4* vec;           // the first vector
  int V, head, nv;

  __device__ __forceinline__ RowView(const void* p, int64_t offset, int V_) {
    base = static_cast<const unsigned char*>(p) + offset * (kBF16 ? 2 : 4);
    V = V_;
    const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(base) & 15u);
    head = mis ? (16 - mis) / (kBF16 ? 2 : 4) : 0;
    if (head > V) head = V;
    nv = (V - head) / G;
    vec = reinterpret_cast<const uint4*>(base + head * (kBF16 ? 2 : 4));
  }
  __device__ __forceinline__ float at(int v) const {
    return kBF16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(base)[v])
                 : reinterpret_cast<const float*>(base)[v];
  }
  // Elements outside the vectors: i in [0, loose()) -> their index.
  __device__ __forceinline__ int loose() const { return V - nv * G; }
  __device__ __forceinline__ int loose_at(int i) const { return i < head ? i : i + nv * G; }
};

__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

template <bool kBF16>
__device__ __forceinline__ uint4 neg_inf_vec() {
  const uint32_t w = kBF16 ? 0xFF80FF80u : 0xFF800000u;
  return make_uint4(w, w, w, w);
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Two fp32 values in one 64-bit register pair (one instruction for both on sm_100 and later).
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Elements 2i and 2i + 1 of a vector (i < G / 2), as fp32.
template <bool kBF16>
__device__ __forceinline__ f32x2 pair_of(const uint4& w, int i) {
  if (kBF16) {
    const uint32_t x = i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
    return pack2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
  }
  return i == 0 ? pack2(__uint_as_float(w.x), __uint_as_float(w.y)) : pack2(__uint_as_float(w.z), __uint_as_float(w.w));
}

// The largest element of a vector (NaN ignored).
template <bool kBF16>
__device__ __forceinline__ float vec_max(const uint4& w) {
  if (kBF16) {
    const __nv_bfloat162 a = __hmax2(reinterpret_cast<const __nv_bfloat162&>(w.x), reinterpret_cast<const __nv_bfloat162&>(w.y));
    const __nv_bfloat162 b = __hmax2(reinterpret_cast<const __nv_bfloat162&>(w.z), reinterpret_cast<const __nv_bfloat162&>(w.w));
    const __nv_bfloat162 m = __hmax2(a, b);
    const uint32_t u = reinterpret_cast<const uint32_t&>(m);
    return fmaxf(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
  }
  return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
}

// A sum of exp(x_v / temperature) in fp32 against a reference logit: s = sum 2^((x_v - ref) c)
// with c = log2(e) / temperature.  The difference is taken before the product, so it is as
// exact at |x| = 1e9 as at 10.  The reference starts where the caller puts it and moves up only
// when a value lies more than 2^64 above it, so a row's threads normally share one reference and
// no element pays for a running maximum.
struct Sum2 {
  float ref, s;
  __device__ __forceinline__ void raise(float to, float c) {  // to > ref
    s *= ex2((ref - to) * c);
    ref = to;
  }
};
constexpr float kRaise = 64.0f;

// The sum of two sums, against the larger reference of those that hold anything.
__device__ __forceinline__ Sum2 merge(const Sum2& a, const Sum2& b, float c) {
  if (b.s == 0.0f) return a;
  if (a.s == 0.0f) return b;
  if (a.ref == b.ref) return Sum2{a.ref, a.s + b.s};
  const float m = fmaxf(a.ref, b.ref);
  return Sum2{m, a.s * ex2((a.ref - m) * c) + b.s * ex2((b.ref - m) * c)};
}

// The warp's sums against the largest reference of those that hold anything; every lane gets the
// same bits (no branch: a butterfly of merge() took ten times as long).
__device__ __forceinline__ Sum2 warp_merge(Sum2 v, float c) {
  float m = v.s == 0.0f ? -FLT_MAX : v.ref;
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float s = v.s == 0.0f ? 0.0f : v.s * ex2((v.ref - m) * c);
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return Sum2{m, s};
}

// Adds the elements of a vector to a sum whose reference is high enough for them.
template <bool kBF16>
__device__ __forceinline__ void add_vec(Sum2& sum, const uint4& w, float c) {
  constexpr int G = kBF16 ? 8 : 4;
  const f32x2 nref = pack2(-sum.ref, -sum.ref), c2 = pack2(c, c);
  f32x2 acc = 0ull;  // two zeros
#pragma unroll
  for (int i = 0; i < G / 2; ++i) {
    float a, b;
    unpack2(mul2(add2(pair_of<kBF16>(w, i), nref), c2), a, b);
    acc = add2(acc, pack2(ex2(a), ex2(b)));
  }
  float a, b;
  unpack2(acc, a, b);
  sum.s += a + b;
}

// A sum against one reference that no element exceeds by much, for the inner loops: a pair of
// partial sums for each pair of a vector, so that a vector adds one term to each.  The exponent
// is one multiply-add, x c - rc with rc the rounded product of the reference and c: what rc's
// rounding left out is put right once, in total().  Only for |rc| <= kFastRef.
constexpr float kFastRef = 0x1p28f;
template <bool kBF16>
struct FastSum {
  static constexpr int kPairs = kBF16 ? 4 : 2;
  f32x2 acc[kPairs], c2, nrc2;
  __device__ __forceinline__ FastSum(float ref, float c) {
    const float rc = ref * c;
    c2 = pack2(c, c);
    nrc2 = pack2(-rc, -rc);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) acc[i] = 0ull;
  }
  __device__ __forceinline__ void add(const uint4& w) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      float a, b;
      unpack2(fma2(pair_of<kBF16>(w, i), c2, nrc2), a, b);
      acc[i] = add2(acc[i], pack2(ex2(a), ex2(b)));
    }
  }
  // The sum of 2^((x - ref) c).
  __device__ __forceinline__ float total(float ref, float c) const {
    f32x2 t = acc[0];
#pragma unroll
    for (int i = 1; i < kPairs; ++i) t = add2(t, acc[i]);
    float a, b, rc, unused;
    unpack2(t, a, b);
    unpack2(nrc2, rc, unused);
    return (a + b) * ex2(-fmaf(ref, c, rc));
  }
};

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A finite reference: differences to it are never inf - inf.
__device__ __forceinline__ float clamp_ref(float x) { return fminf(fmaxf(x, -FLT_MAX), FLT_MAX); }

// ---- bulk copies between global and shared memory (16-byte addresses and sizes) -----------------
__device__ __forceinline__ uint32_t shared_u32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
// A barrier for one copy; visible to the copy engine and, after a block barrier, to the block.
__device__ __forceinline__ void copy_barrier_init(unsigned long long* bar) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(shared_u32(bar)) : "memory");
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void expect_bytes(unsigned long long* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(shared_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_in(void* dst, const void* src, uint32_t bytes, unsigned long long* bar) {
  expect_bytes(bar, bytes);
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   shared_u32(dst)),
               "l"(src), "r"(bytes), "r"(shared_u32(bar))
               : "memory");
}
// Stores v to *to in the shared memory of the cluster's CTA `cta`, counted at its barrier *bar.
__device__ __forceinline__ void send_float(float* to, float v, unsigned long long* bar, int cta) {
  uint32_t ra, rb;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(shared_u32(to)), "r"(cta));
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(rb) : "r"(shared_u32(bar)), "r"(cta));
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(ra), "r"(__float_as_uint(v)),
               "r"(rb)
               : "memory");
}
// Waits for the copy, for about two seconds at most; false when it has not landed by then.
__device__ __forceinline__ bool copy_landed(unsigned long long* bar) {
  const long long t0 = clock64();
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], 0;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(shared_u32(bar))
        : "memory");
    if (ok) return true;
    if (clock64() - t0 > 4000000000LL) return false;
  }
}
// Before a block barrier after which one thread stores what the block wrote to shared memory.
__device__ __forceinline__ void publish_to_copies() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// The store, by one thread, which waits until the shared memory has been read.
__device__ __forceinline__ void copy_out(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(shared_u32(src)), "r"(bytes)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

}  // namespace stream
}  // namespace kps
