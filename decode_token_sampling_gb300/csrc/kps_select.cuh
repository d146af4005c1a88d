// kps_select.cuh — the first elements of a row's order (value descending, index ascending; NaN counts as
// -inf): keys, counts by digits and the exact selection over a whole row.  Shared by the kernels that list
// a row's top logits.
#pragma once

#include "kps_stream.cuh"

namespace kps {
namespace select {

using namespace stream;

constexpr int kNT = 256;  // threads per CTA, unless a template says otherwise (NT)
constexpr int kNW = kNT / 32;
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;

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

// Every element of the row, with the warp converged: f(valid, value, index).
template <bool kBF16, int NT = kNT, class F>
__device__ __forceinline__ void each_raw(const RowView<kBF16>& x, F&& f) {
  constexpr int G = kBF16 ? 8 : 4, kU = 6;  // loads in flight
  for (int base = 0; base < x.nv; base += NT * kU) {
    uint4 w[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int g = base + u * NT + static_cast<int>(threadIdx.x);
      w[u] = g < x.nv ? ld_stream(x.vec + g) : neg_inf_vec<kBF16>();
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int g = base + u * NT + static_cast<int>(threadIdx.x);
#pragma unroll
      for (int e = 0; e < G; ++e) f(g < x.nv, elem<kBF16>(w[u], e), x.head + g * G + e);
    }
  }
  const bool in = static_cast<int>(threadIdx.x) < x.loose();
  const int v = in ? x.loose_at(threadIdx.x) : 0;
  f(in, in ? x.at(v) : -INFINITY, v);
}
// The same with NaN as -inf.
template <bool kBF16, int NT = kNT, class F>
__device__ __forceinline__ void each(const RowView<kBF16>& x, F&& f) {
  each_raw<kBF16, NT>(x, [&](bool valid, float y, int v) { f(valid, clean(y), v); });
}

// The exact selection, by one CTA, for rows whose list came out too short or too long: the n-th
// element of the order by 8-bit digits of its key and, among equal keys, of its index; then the n
// elements as survivors and the thread's sum of all others.  At least n elements have a key of
// floor or more.
template <bool kBF16, int NT = kNT, class S>
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
      for (int i = threadIdx.x; i < 256; i += NT) sm.hist[i] = 0u;
      __syncthreads();
      each<kBF16, NT>(x, [&](bool valid, float y, int v) {
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
  each<kBF16, NT>(x, [&](bool valid, float y, int v) {
    const unsigned long long w = word_of(fkey(y), v);
    if (valid && n > 0 && w >= at) {
      sm.words[atomicAdd(&sm.n_words, 1u)] = w;  // n of them
    } else if (valid) {
      add_one(sum, y, c);
    }
  });
  return sum;
}

}  // namespace select
}  // namespace kps
