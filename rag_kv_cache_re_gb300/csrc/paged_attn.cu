// Attention of a batch of sequences over a shared prefix and their own tokens, both in pages.
#include <algorithm>
#include <cmath>

#include "paged.cuh"

namespace qcf {

struct AttnArgs {
  const void* q;
  int64_t q_stride;
  const void* k;
  const void* v;
  void* o;
  float* lse;
  int Hq;
  float scale_log2;
};

// One warp per (row, query head).  32 keys at a time: lane j scores key j against the row held
// in registers, the warp shares the maximum and the sum, then lanes take D / 32 output entries
// each and add the keys' values.  The keys of the prefix come first, then the own ones.
template <typename T, int D>
__global__ void __launch_bounds__(256) paged_attn_kernel(const PagedView c, const BatchView b, const AttnArgs a,
                                                         unsigned int* status) {
  constexpr int E = D / 32 > 0 ? D / 32 : 1;   // output entries per lane: e + E lane
  const int w = static_cast<int>((static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5), lane = threadIdx.x & 31;
  const int row = w / a.Hq, h = w - row * a.Hq;
  if (row >= b.n_rows) return;
  const int seq = warp_seq_of_row(b, row);
  if (seq < 0) return;
  const SeqSpan s = seq_span(b, seq);
  if (s.bad) {
    if (lane == 0) flag_status(status, QCF_DEV_BAD_INDEX);
    return;
  }
  if (row >= s.row0 + s.nq) return;
  const int keys[2] = {b.prefix_len, s.len - s.nq + (row - s.row0) + 1};
  const int32_t* pages[2] = {b.prefix_pages, b.page_table + static_cast<int64_t>(seq) * b.table_stride};
  const int64_t head = static_cast<int64_t>(h / (a.Hq / c.Hkv)) * c.head_stride;
  const T* q = static_cast<const T*>(a.q) + row * a.q_stride + h * D;
  const T* K = static_cast<const T*>(a.k) + head;
  const T* V = static_cast<const T*>(a.v) + head;
  float m = -INFINITY, l = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int part = 0; part < 2; ++part) {
    for (int j0 = 0; j0 < keys[part]; j0 += 32) {
      const int j = j0 + lane;
      int64_t slot = -1;
      if (j < keys[part]) {
        slot = slot_of(c, pages[part], j);
        if (slot < 0) flag_status(status, QCF_DEV_BAD_INDEX);
      }
      float x = -INFINITY;
      if (slot >= 0) {
        x = 0.f;
        for (int d = 0; d < D; d += 8) {
          const Vec<T, 8> kv = *reinterpret_cast<const Vec<T, 8>*>(K + slot + d);
          const Vec<T, 8> qv = *reinterpret_cast<const Vec<T, 8>*>(q + d);
#pragma unroll
          for (int e = 0; e < 8; ++e) x = fmaf(to_f32(qv.v[e]), to_f32(kv.v[e]), x);
        }
        x *= a.scale_log2;
      }
      float top = x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float mn = fmaxf(m, top);
      if (mn == -INFINITY) continue;
      const float f = exp2f(m - mn), p = exp2f(x - mn);
      m = mn;
      l = l * f + p;   // this lane's share; the lanes meet at the end
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= f;
      const int n = min(32, keys[part] - j0);
      for (int i = 0; i < n; ++i) {
        const float pi = __shfl_sync(0xffffffffu, p, i);
        const int64_t si = __shfl_sync(0xffffffffu, slot, i);
        if (si < 0) continue;
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (lane * E + e < D) acc[e] = fmaf(pi, to_f32(V[si + lane * E + e]), acc[e]);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const int64_t out = static_cast<int64_t>(row) * a.Hq + h;
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (lane * E + e < D) static_cast<T*>(a.o)[out * D + lane * E + e] = from_f32<T>(acc[e] * inv);
  if (a.lse && lane == 0) a.lse[out] = (m + log2f(l)) * 0.69314718055994531f;
}

template <typename T, int D>
static cudaError_t shared_prefix_attn_launch(const PagedView& c, const BatchView& b, const AttnArgs& a, cudaStream_t st) {
  LaunchScope ls(KC_OWN_ATTN, st);
  const int64_t warps = static_cast<int64_t>(b.n_rows) * a.Hq;
  paged_attn_kernel<T, D><<<static_cast<unsigned>((warps + 7) / 8), 256, 0, st>>>(c, b, a, device_status_ptr());
  return cudaGetLastError();
}

template <typename T>
static cudaError_t shared_prefix_attn_type(const PagedView& c, const BatchView& b, const AttnArgs& a, cudaStream_t st) {
  switch (c.D) {
    case 16: return shared_prefix_attn_launch<T, 16>(c, b, a, st);
    case 64: return shared_prefix_attn_launch<T, 64>(c, b, a, st);
    default: return shared_prefix_attn_launch<T, 128>(c, b, a, st);
  }
}

static qcf_status check_attn(const char* who, const qcf_paged_kv* cache, const qcf_paged_batch* batch, int Hq, PagedView* c,
                             BatchView* b) {
  const qcf_status s = check_paged(who, cache, batch, c, b);
  if (s != QCF_OK) return s;
  if (Hq <= 0 || Hq % c->Hkv || Hq / c->Hkv > 16) return set_error(QCF_ERR_SHAPE, "%s: Hq=%d Hkv=%d", who, Hq, c->Hkv);
  if (static_cast<int64_t>(b->n_rows) * Hq > INT32_MAX / 128)
    return set_error(QCF_ERR_SHAPE, "%s: %d rows of %d heads are too many for one call", who, b->n_rows, Hq);
  return QCF_OK;
}

}  // namespace qcf

using namespace qcf;

extern "C" {

size_t qcf_shared_prefix_attn_workspace_size(const qcf_paged_kv* cache, const qcf_paged_batch* batch, int Hq) {
  PagedView c;
  BatchView b;
  if (check_attn("qcf_shared_prefix_attn_workspace_size", cache, batch, Hq, &c, &b) != QCF_OK) return 0;
  return 0;
}

qcf_status qcf_shared_prefix_attn(const qcf_paged_kv* cache, const qcf_paged_batch* batch, const void* q, int64_t q_stride,
                                  int Hq, float scale, void* o, float* lse, void* ws, size_t ws_bytes, void* stream) {
  const char* who = "qcf_shared_prefix_attn";
  PagedView c;
  BatchView b;
  const qcf_status s = check_attn(who, cache, batch, Hq, &c, &b);
  if (s != QCF_OK) return s;
  if (!q || !o) return set_error(QCF_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (!(scale > 0.f) || !std::isfinite(scale)) return set_error(QCF_ERR_INVALID_ARG, "%s: scale=%g", who, scale);
  if (q_stride < static_cast<int64_t>(Hq) * c.D)
    return set_error(QCF_ERR_SHAPE, "%s: q_stride %lld for %d x %d entries", who, (long long)q_stride, Hq, c.D);
  if (take_fault(4) || !aligned16(q) || !aligned16(o) || q_stride % 8 || (reinterpret_cast<uintptr_t>(ws) & 255u))
    return set_error(QCF_ERR_ALIGN, "%s: pointers and strides must be multiples of 16 bytes, ws of 256", who);
  if (take_fault(1)) return set_error(QCF_ERR_INVALID_ARG, "%s: injected invalid index table", who);
  if (take_fault(2) || ws_bytes < qcf_shared_prefix_attn_workspace_size(cache, batch, Hq))
    return set_error(QCF_ERR_WORKSPACE, "%s: workspace too small", who);
  if (b.n_seq == 0 || b.n_rows == 0) return QCF_OK;
  const AttnArgs a{q, q_stride, cache->k, cache->v, o, lse, Hq, scale * 1.4426950408889634f};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = cache->dtype == QCF_BF16 ? shared_prefix_attn_type<__nv_bfloat16>(c, b, a, st)
                                                 : shared_prefix_attn_type<__half>(c, b, a, st);
  return e == cudaSuccess ? QCF_OK : cuda_error(e, "qcf_shared_prefix_attn: launch");
}

}  // extern "C"
