// Rotation of head entries shared by the rotary and the paged-append kernels.
#pragma once

#include <cuda_fp16.h>

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
template <int V>
__device__ __forceinline__ ItemAt item_at(int item, int R, bool interleaved) {
  const int k = item * V;
  ItemAt it;
  it.turns = k < R / 2;
  if (it.turns && !interleaved) {
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

template <typename T, int V>
__device__ __forceinline__ void turn_item(Vec<T, V>& x, Vec<T, V>& y, const Angles<V>& g, bool interleaved) {
  if (interleaved) {   // pairs (x0, x1), .. then (y0, y1), ..: a V of 1 keeps its one pair in x, y
    if constexpr (V == 1) {
      float oa, ob;
      turn(to_f32(x.v[0]), to_f32(y.v[0]), g.c[0], g.s[0], oa, ob);
      x.v[0] = from_f32<T>(oa);
      y.v[0] = from_f32<T>(ob);
    } else {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        float oa, ob;
        turn(to_f32(x.v[2 * i]), to_f32(x.v[2 * i + 1]), g.c[i], g.s[i], oa, ob);
        x.v[2 * i] = from_f32<T>(oa);
        x.v[2 * i + 1] = from_f32<T>(ob);
        turn(to_f32(y.v[2 * i]), to_f32(y.v[2 * i + 1]), g.c[V / 2 + i], g.s[V / 2 + i], oa, ob);
        y.v[2 * i] = from_f32<T>(oa);
        y.v[2 * i + 1] = from_f32<T>(ob);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float oa, ob;
      turn(to_f32(x.v[i]), to_f32(y.v[i]), g.c[i], g.s[i], oa, ob);
      x.v[i] = from_f32<T>(oa);
      y.v[i] = from_f32<T>(ob);
    }
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
