// Rotation of head entries shared by the rotary and the paged-append kernels.
#pragma once

#include <cuda_fp16.h>
#include <string.h>

#include <type_traits>

#include "qcf_internal.cuh"

namespace qcf {

// N elements of T moved in accesses of at most 16 bytes; addresses are N-element aligned.
template <typename T, int N>
struct alignas(sizeof(T) * N < 16 ? sizeof(T) * N : 16) Vec {
  T v[N];
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

// One item of a head: V pairs that turn (item < R / 2 / V), or 2 V entries behind the
// rotated width that are copied.  A head of D entries has D / 2 / V items; V divides R / 2
// and (D - R) / 2.  Both runs of V entries of an item are contiguous:
//   half layout   entries k .. k + V - 1 and R/2 + k ..     with k = item V
//   interleaved   entries 2k .. 2k + 2V - 1, pairs side by side
//   copied        entries R + 2 (k - R/2) ..
struct ItemAt {
  int a, b;     // first entries of the two runs
  bool turns;
};
template <int V, bool INTER>
__device__ __forceinline__ ItemAt item_at(int item, int R) {
  const int k = item * V;
  ItemAt it;
  it.turns = k < R / 2;
  if (it.turns && !INTER) {
    it.a = k;
    it.b = R / 2 + k;
  } else {
    it.a = 2 * k;   // for a copied item too: R + 2 (k - R/2) = 2k
    it.b = 2 * k + V;
  }
  return it;
}

template <int V>
struct Angles {
  float c[V], s[V];
};
template <int V>
__device__ __forceinline__ Angles<V> load_angles(const float* __restrict__ cos_t, const float* __restrict__ sin_t, int pos,
                                                 int R, int item, bool inverse) {
  Angles<V> g;
  const size_t at = static_cast<size_t>(pos) * (R / 2) + item * V;
  const Vec<float, V> c = *reinterpret_cast<const Vec<float, V>*>(cos_t + at);
  const Vec<float, V> s = *reinterpret_cast<const Vec<float, V>*>(sin_t + at);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    g.c[i] = c.v[i];
    g.s[i] = inverse ? -s.v[i] : s.v[i];
  }
  return g;
}

// (a, b) -> (a cos - b sin, b cos + a sin); every product and sum rounded on its own (no
// contraction into FMAs), the arithmetic of the kernels that re-rotate stored keys.
__device__ __forceinline__ void turn(float a, float b, float c, float s, float& oa, float& ob) {
  oa = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  ob = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

// V entries as they lie in memory: 32-bit words (two 16-bit entries each) kept whole until they are
// turned, so that a run of 8 waits in four registers.
template <typename T, int V>
struct Run {
  static constexpr int BYTES = sizeof(T) * V;
  using Word = typename std::conditional<BYTES % 4 == 0, uint32_t, uint16_t>::type;
  static constexpr int N = BYTES / sizeof(Word);
  Vec<Word, N> w;
  __device__ __forceinline__ void load(const T* p) { w = *reinterpret_cast<const Vec<Word, N>*>(p); }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<Vec<Word, N>*>(p) = w; }
};
__device__ __forceinline__ float2 unpack2(uint32_t w, __nv_bfloat16) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 unpack2(uint32_t w, __half) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
__device__ __forceinline__ uint32_t repack2(float lo, float hi, __nv_bfloat16) { return pack_bf16x2(lo, hi); }
__device__ __forceinline__ uint32_t repack2(float lo, float hi, __half) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Turns the pairs of one item: x and y are its two runs.
template <typename T, int V, bool INTER>
__device__ __forceinline__ void turn_item(Run<T, V>& x, Run<T, V>& y, const Angles<V>& g) {
  if constexpr (sizeof(T) == 2 && V >= 2) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 p = unpack2(x.w.v[i], T()), q = unpack2(y.w.v[i], T());
      float2 a, b;
      if constexpr (INTER) {   // a word is a pair; the pairs of x come before those of y
        turn(p.x, p.y, g.c[i], g.s[i], a.x, a.y);
        turn(q.x, q.y, g.c[V / 2 + i], g.s[V / 2 + i], b.x, b.y);
      } else {
        turn(p.x, q.x, g.c[2 * i], g.s[2 * i], a.x, b.x);
        turn(p.y, q.y, g.c[2 * i + 1], g.s[2 * i + 1], a.y, b.y);
      }
      x.w.v[i] = repack2(a.x, a.y, T());
      y.w.v[i] = repack2(b.x, b.y, T());
    }
  } else {
    T e[2 * V];
    memcpy(e, &x, sizeof(T) * V);
    memcpy(e + V, &y, sizeof(T) * V);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int ia = INTER ? 2 * i : i, ib = INTER ? 2 * i + 1 : V + i;
      float a, b;
      turn(to_f32(e[ia]), to_f32(e[ib]), g.c[i], g.s[i], a, b);
      e[ia] = from_f32<T>(a);
      e[ib] = from_f32<T>(b);
    }
    memcpy(&x, e, sizeof(T) * V);
    memcpy(&y, e + V, sizeof(T) * V);
  }
}

// Pairs per item: the widest of 8, 4, 2, 1 that divides both parts of the head and the row
// strides, so that the runs of an item stay whole and aligned (16-byte accesses for 16-bit
// types whenever R / 2, (D - R) / 2 and the strides are multiples of 8).
inline int item_width(int R, int D, int64_t stride_a = 0, int64_t stride_b = 0) {
  for (int v = 8; v > 1; v /= 2)
    if ((R / 2) % v == 0 && ((D - R) / 2) % v == 0 && stride_a % v == 0 && stride_b % v == 0) return v;
  return 1;
}

}  // namespace qcf
