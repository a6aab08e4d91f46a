// Attention of many new tokens of a sequence at a time: whole prompts packed one behind the other,
// and chunks of prompts over a paged cache that holds them already.
//
// For a row at position p, o = sum_j w_j V_j / sum_j w_j with w_j = 2^(x_j - m), x_j = scale log2(e) q.K_j over
// the keys j <= p (and j > p - window), m a running maximum: one pass over the keys, the sums rescaled
// when m grows.
//
// A CTA takes 64 score rows (new rows x the G query heads of one KV head) of one sequence, 16 to a
// warp, and walks the key tiles that any of them sees; products on warp tensor cores.
#include <algorithm>
#include <cmath>

#include "paged_attn.cuh"

namespace qcf {

constexpr int kMaxChunkSeqs = 16384;
constexpr int kChunkRows = 64, kChunkKeys = 64;

// What the two entry points differ in: keys and values as rows of one tensor each, or in pages.
struct ChunkArgs {
  AttnArgs a;
  const void* k;
  const void* v;
  int64_t kv_stride;   // packed: entries from row to row
  int D, window;
};

__device__ __forceinline__ SeqSpan chunk_span(const BatchView& b, int seq) {
  if (b.kv_len) return seq_span(b, seq);
  SeqSpan s;
  s.row0 = b.row_start[seq];
  const int end = b.row_start[seq + 1];
  s.bad = s.row0 < 0 || end < s.row0 || end > b.n_rows || end - s.row0 > b.max_q;
  s.nq = s.len = s.bad ? 0 : end - s.row0;
  return s;
}

template <typename T, int DP, bool PAGED>
__global__ void __launch_bounds__(128) chunk_attn_kernel(const PagedView c, const BatchView b, const ChunkArgs p, unsigned int* status) {
  constexpr int ROW = DP + 8;   // 16 bytes more than a row: eight rows lie in different banks
  constexpr unsigned kAll = 0xffffffffu;
  __shared__ __align__(16) T ks[kChunkKeys * ROW], vs[kChunkKeys * ROW];
  __shared__ unsigned long long gone_s;
  __shared__ int unit_s[2];
  const AttnArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = blockIdx.x / c.Hkv, g = blockIdx.x - unit * c.Hkv;
  if (warp == 0) {   // the sequence and row block of this unit
    int before = 0, seq = -1, block = 0;
    for (int s0 = 0; s0 < b.n_seq; s0 += 32) {
      int n = 0;
      if (s0 + lane < b.n_seq) {
        const SeqSpan s = chunk_span(b, s0 + lane);
        if (s.bad && blockIdx.x == 0) flag_status(status, QCF_DEV_BAD_INDEX);
        n = (s.nq * a.G + kChunkRows - 1) / kChunkRows;
      }
      int run = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kAll, run, o);
        if (lane >= o) run += v;
      }
      const unsigned hit = __ballot_sync(kAll, n > 0 && unit >= before + run - n && unit < before + run);
      if (hit && seq < 0) {
        seq = s0 + __ffs(hit) - 1;
        block = unit - before - __shfl_sync(kAll, run - n, seq - s0);
      }
      before += __shfl_sync(kAll, run, 31);
      if (seq >= 0 && blockIdx.x > 0) break;
    }
    if (lane == 0) {
      unit_s[0] = seq;
      unit_s[1] = block;
    }
  }
  __syncthreads();
  const int seq = unit_s[0];
  if (seq < 0) return;
  const SeqSpan s = chunk_span(b, seq);
  const int rho0 = unit_s[1] * kChunkRows, end = min(rho0 + kChunkRows, s.nq * a.G);
  const int r_lo = rho0 + warp * 16 + (lane >> 2), r_hi = r_lo + 8, qc = (lane & 3) * 2;
  const int prefix = b.prefix_len, old = prefix + s.len - s.nq;   // position of the first new row
  const int i_lo = min(r_lo, end - 1) / a.G, i_hi = min(r_hi, end - 1) / a.G;
  const int p_lo = old + i_lo, p_hi = old + i_hi;
  const int first = p.window ? max(0, old + rho0 / a.G - p.window + 1) : 0, last = old + (end - 1) / a.G;
  const int low_lo = p.window ? p_lo - p.window : -1, low_hi = p.window ? p_hi - p.window : -1;

  uint32_t qf[DP / 16][4];
  {
    const T* ql = static_cast<const T*>(a.q) + (s.row0 + i_lo) * a.q_stride + static_cast<int64_t>(g * a.G + min(r_lo, end - 1) - i_lo * a.G) * p.D;
    const T* qh = static_cast<const T*>(a.q) + (s.row0 + i_hi) * a.q_stride + static_cast<int64_t>(g * a.G + min(r_hi, end - 1) - i_hi * a.G) * p.D;
#pragma unroll
    for (int t = 0; t < DP / 16; ++t) {
      const int col = t * 16 + qc;
      qf[t][0] = col < p.D ? *reinterpret_cast<const uint32_t*>(ql + col) : 0u;
      qf[t][1] = col < p.D ? *reinterpret_cast<const uint32_t*>(qh + col) : 0u;
      qf[t][2] = col + 8 < p.D ? *reinterpret_cast<const uint32_t*>(ql + col + 8) : 0u;
      qf[t][3] = col + 8 < p.D ? *reinterpret_cast<const uint32_t*>(qh + col + 8) : 0u;
    }
  }

  constexpr float kLift = kWeightLift<T>;
  float m_lo = -INFINITY, m_hi = -INFINITY, l_lo = 0.f, l_hi = 0.f;
  float acc[DP / 8][4];
#pragma unroll
  for (int i = 0; i < DP / 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  const int mi = lane >> 3, mr = lane & 7;
  const uint32_t ka = smem_u32(ks), va = smem_u32(vs);
  for (int t0 = first / kChunkKeys * kChunkKeys; t0 <= last; t0 += kChunkKeys) {
    __syncthreads();
    if (threadIdx.x == 0) gone_s = 0;
    __syncthreads();
    for (int e = threadIdx.x; e < kChunkKeys * (DP / 8); e += 128) {
      const int key = e / (DP / 8), col = e % (DP / 8) * 8, j = t0 + key;
      uint4 kv = make_uint4(0u, 0u, 0u, 0u), vv = kv;
      int64_t at = -1;
      if (j < prefix + s.len) {
        if constexpr (PAGED) {
          at = j < prefix ? slot_of(c, b.prefix_pages, j) : slot_of(c, b.page_table + static_cast<int64_t>(seq) * b.table_stride, j - prefix);
          if (at < 0 && col == 0) {
            atomicOr(&gone_s, 1ull << key);
            flag_status(status, QCF_DEV_BAD_INDEX);
          }
          if (at >= 0) at += g * c.head_stride;
        } else {
          at = (s.row0 + j) * p.kv_stride + static_cast<int64_t>(g) * p.D;
        }
      }
      if (at >= 0 && col < p.D) {
        kv = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.k) + at + col);
        vv = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.v) + at + col);
      }
      *reinterpret_cast<uint4*>(ks + key * ROW + col) = kv;
      *reinterpret_cast<uint4*>(vs + key * ROW + col) = vv;
    }
    __syncthreads();
    const unsigned long long gone = gone_s;
    float sc[kChunkKeys / 8][4];
#pragma unroll
    for (int j = 0; j < kChunkKeys / 8; ++j) sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
#pragma unroll
    for (int t = 0; t < DP / 16; ++t)
#pragma unroll
      for (int h = 0; h < kChunkKeys / 16; ++h) {
        uint32_t b0, b1, b2, b3;
        ldsm_x4(ka + ((h * 16 + (mi >> 1) * 8 + mr) * ROW + t * 16 + (mi & 1) * 8) * 2, b0, b1, b2, b3);
        mma_16816<T>(sc[2 * h], qf[t], b0, b1);
        mma_16816<T>(sc[2 * h + 1], qf[t], b2, b3);
      }
    float top_lo = -INFINITY, top_hi = -INFINITY;
#pragma unroll
    for (int j = 0; j < kChunkKeys / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int key = t0 + j * 8 + qc + (e & 1);
        if (key > (e < 2 ? p_lo : p_hi) || key <= (e < 2 ? low_lo : low_hi) || (gone >> (key - t0) & 1)) sc[j][e] = -INFINITY;
        if (e < 2) top_lo = fmaxf(top_lo, sc[j][e]); else top_hi = fmaxf(top_hi, sc[j][e]);
      }
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
      top_lo = fmaxf(top_lo, __shfl_xor_sync(kAll, top_lo, o));
      top_hi = fmaxf(top_hi, __shfl_xor_sync(kAll, top_hi, o));
    }
    const float n_lo = fmaxf(m_lo, top_lo * a.scale_log2 - kLift), n_hi = fmaxf(m_hi, top_hi * a.scale_log2 - kLift);
    const float f_lo = m_lo == -INFINITY ? 0.f : fast_exp2(m_lo - n_lo), f_hi = m_hi == -INFINITY ? 0.f : fast_exp2(m_hi - n_hi);
    m_lo = n_lo;
    m_hi = n_hi;
    l_lo *= f_lo;
    l_hi *= f_hi;
#pragma unroll
    for (int j = 0; j < DP / 8; ++j) {
      acc[j][0] *= f_lo;
      acc[j][1] *= f_lo;
      acc[j][2] *= f_hi;
      acc[j][3] *= f_hi;
    }
    const float b_lo = m_lo == -INFINITY ? 0.f : -m_lo, b_hi = m_hi == -INFINITY ? 0.f : -m_hi;
#pragma unroll
    for (int j = 0; j < kChunkKeys / 8; ++j) {
      sc[j][0] = fast_exp2(fmaf(sc[j][0], a.scale_log2, b_lo));
      sc[j][1] = fast_exp2(fmaf(sc[j][1], a.scale_log2, b_lo));
      sc[j][2] = fast_exp2(fmaf(sc[j][2], a.scale_log2, b_hi));
      sc[j][3] = fast_exp2(fmaf(sc[j][3], a.scale_log2, b_hi));
      l_lo += sc[j][0] + sc[j][1];
      l_hi += sc[j][2] + sc[j][3];
    }
    // the weights meet the values in the 16-bit type of both (the MMA's); their sum stays fp32
#pragma unroll
    for (int h = 0; h < kChunkKeys / 16; ++h) {
      const uint32_t pa[4] = {pack2<T>(sc[2 * h][0], sc[2 * h][1]), pack2<T>(sc[2 * h][2], sc[2 * h][3]),
                              pack2<T>(sc[2 * h + 1][0], sc[2 * h + 1][1]), pack2<T>(sc[2 * h + 1][2], sc[2 * h + 1][3])};
#pragma unroll
      for (int dp = 0; dp < DP / 16; ++dp) {
        uint32_t b0, b1, b2, b3;
        ldsm_x4_t(va + ((h * 16 + (mi & 1) * 8 + mr) * ROW + dp * 16 + (mi >> 1) * 8) * 2, b0, b1, b2, b3);
        mma_16816<T>(acc[2 * dp], pa, b0, b1);
        mma_16816<T>(acc[2 * dp + 1], pa, b2, b3);
      }
    }
  }
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    l_lo += __shfl_xor_sync(kAll, l_lo, o);
    l_hi += __shfl_xor_sync(kAll, l_hi, o);
  }
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int rho = half ? r_hi : r_lo;
    if (rho >= end) continue;
    const float m = half ? m_hi : m_lo, l = half ? l_hi : l_lo, inv = l == 0.f ? 0.f : 1.f / l;
    const int i = half ? i_hi : i_lo;
    const int64_t place = static_cast<int64_t>(s.row0 + i) * a.Hq + g * a.G + rho - i * a.G;
    T* o = static_cast<T*>(a.o) + place * p.D;
#pragma unroll
    for (int j = 0; j < DP / 8; ++j)
      if (j * 8 + qc < p.D) *reinterpret_cast<uint32_t*>(o + j * 8 + qc) = pack2<T>(acc[j][2 * half] * inv, acc[j][2 * half + 1] * inv);
    if (a.lse && qc == 0) a.lse[place] = (m + log2f(l)) * 0.69314718055994531f;
  }
}

// ------------------------------------------------------------------ host

// Row blocks of a KV head at most: every sequence may end with a part of one.
static int64_t most_blocks(const BatchView& b, int G) {
  const int64_t rows = std::min(b.max_q, b.n_rows);
  return std::min(b.n_seq * ((rows * G + kChunkRows - 1) / kChunkRows),
                  (static_cast<int64_t>(b.n_rows) * G + static_cast<int64_t>(b.n_seq) * (kChunkRows - 1)) / kChunkRows);
}

template <typename T, bool PAGED>
static cudaError_t chunk_launch(const PagedView& c, const BatchView& b, const ChunkArgs& p, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(std::max<int64_t>(1, most_blocks(b, p.a.G)) * c.Hkv));
  LaunchScope ls(KC_CHUNK_ATTN, st);
  if (p.D <= 64)
    chunk_attn_kernel<T, 64, PAGED><<<grid, 128, 0, st>>>(c, b, p, device_status_ptr());
  else
    chunk_attn_kernel<T, 128, PAGED><<<grid, 128, 0, st>>>(c, b, p, device_status_ptr());
  return cudaGetLastError();
}

static qcf_status check_sizes(const char* who, const PagedView& c, const BatchView& b, int Hq) {
  if (b.n_seq > kMaxChunkSeqs) return set_error(QCF_ERR_SHAPE, "%s: n_seq=%d (at most %d)", who, b.n_seq, kMaxChunkSeqs);
  if (Hq <= 0 || Hq % c.Hkv || Hq / c.Hkv > 128) return set_error(QCF_ERR_SHAPE, "%s: Hq=%d Hkv=%d", who, Hq, c.Hkv);
  if (static_cast<int64_t>(b.n_rows) * Hq > INT32_MAX / 128)
    return set_error(QCF_ERR_SHAPE, "%s: %d rows of %d heads are too many for one call", who, b.n_rows, Hq);
  return QCF_OK;
}

static qcf_status check_packed(const char* who, int n_seq, int n_rows, int max_len, int Hq, int Hkv, int D, PagedView* c, BatchView* b) {
  if (n_seq < 0 || n_rows < 0 || max_len < 0)
    return set_error(QCF_ERR_SHAPE, "%s: n_seq=%d n_rows=%d max_len=%d", who, n_seq, n_rows, max_len);
  if (Hkv <= 0 || Hkv > 65535 || D < 8 || D > 128 || D % 8) return set_error(QCF_ERR_SHAPE, "%s: Hkv=%d D=%d", who, Hkv, D);
  *c = PagedView{};
  c->Hkv = Hkv;
  c->D = D;
  *b = BatchView{};
  b->n_seq = n_seq;
  b->n_rows = n_rows;
  b->max_q = b->max_len = std::min(max_len, n_rows);
  return check_sizes(who, *c, *b, Hq);
}

// The arguments that both calls have, and their injected faults.
static qcf_status check_chunk(const char* who, const PagedView& c, const void* q, int64_t q_stride, int Hq, float scale, int window, void* o,
                              void* ws) {
  if (!q || !o) return set_error(QCF_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (!(scale > 0.f) || !std::isfinite(scale * 1.4426950408889634f)) return set_error(QCF_ERR_INVALID_ARG, "%s: scale=%g", who, scale);
  if (window < 0) return set_error(QCF_ERR_INVALID_ARG, "%s: window=%d", who, window);
  if (q_stride < static_cast<int64_t>(Hq) * c.D)
    return set_error(QCF_ERR_SHAPE, "%s: q_stride %lld for %d x %d entries", who, (long long)q_stride, Hq, c.D);
  if (take_fault(4) || !aligned16(q) || !aligned16(o) || q_stride % 8 || (reinterpret_cast<uintptr_t>(ws) & 255u))
    return set_error(QCF_ERR_ALIGN, "%s: pointers and strides must be multiples of 16 bytes, ws of 256", who);
  // finished rows of o are written while the queries of others are still read
  if (o == q && q_stride != static_cast<int64_t>(Hq) * c.D)
    return set_error(QCF_ERR_SHAPE, "%s: o is q, whose rows lie %lld entries apart instead of %d x %d", who, (long long)q_stride, Hq, c.D);
  if (take_fault(1)) return set_error(QCF_ERR_INVALID_ARG, "%s: injected invalid index table", who);
  if (take_fault(2)) return set_error(QCF_ERR_WORKSPACE, "%s: injected short workspace", who);
  return QCF_OK;
}

static AttnArgs attn_args(const void* q, int64_t q_stride, void* o, float* lse, int Hq, int Hkv, float scale) {
  const int G = Hq / Hkv;
  return AttnArgs{q, q_stride, o, lse, Hq, G, static_cast<uint32_t>(((1ull << 32) + G - 1) / G), scale * 1.4426950408889634f};
}

}  // namespace qcf

using namespace qcf;

extern "C" {

size_t qcf_packed_causal_attn_workspace_size(int n_seq, int n_rows, int max_len, int Hq, int Hkv, int D) {
  PagedView c;
  BatchView b;
  check_packed("qcf_packed_causal_attn_workspace_size", n_seq, n_rows, max_len, Hq, Hkv, D, &c, &b);
  return 0;
}

qcf_status qcf_packed_causal_attn(const void* q, int64_t q_stride, const void* k, const void* v, int64_t kv_stride, int dtype,
                                  const int32_t* row_start, int n_seq, int n_rows, int max_len, int Hq, int Hkv, int D, float scale,
                                  int window, void* o, float* lse, void* ws, size_t ws_bytes, void* stream) {
  const char* who = "qcf_packed_causal_attn";
  PagedView c;
  BatchView b;
  qcf_status s = check_packed(who, n_seq, n_rows, max_len, Hq, Hkv, D, &c, &b);
  if (s != QCF_OK) return s;
  if (!k || !v || !row_start) return set_error(QCF_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (dtype != QCF_BF16 && dtype != QCF_F16) return set_error(QCF_ERR_INVALID_ARG, "%s: dtype %d", who, dtype);
  if (kv_stride < static_cast<int64_t>(Hkv) * D)
    return set_error(QCF_ERR_SHAPE, "%s: kv_stride %lld for %d x %d entries", who, (long long)kv_stride, Hkv, D);
  if (!aligned16(k) || !aligned16(v) || kv_stride % 8)
    return set_error(QCF_ERR_ALIGN, "%s: pointers and strides must be multiples of 16 bytes", who);
  if ((s = check_chunk(who, c, q, q_stride, Hq, scale, window, o, ws)) != QCF_OK) return s;
  if (n_seq == 0 || n_rows == 0) return QCF_OK;
  b.row_start = row_start;
  const ChunkArgs p{attn_args(q, q_stride, o, lse, Hq, Hkv, scale), k, v, kv_stride, D, window};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == QCF_BF16 ? chunk_launch<__nv_bfloat16, false>(c, b, p, st) : chunk_launch<__half, false>(c, b, p, st);
  return e == cudaSuccess ? QCF_OK : cuda_error(e, "qcf_packed_causal_attn: launch");
}

size_t qcf_paged_chunk_attn_workspace_size(const qcf_paged_kv* cache, const qcf_paged_batch* batch, int Hq) {
  const char* who = "qcf_paged_chunk_attn_workspace_size";
  PagedView c;
  BatchView b;
  if (check_paged(who, cache, batch, &c, &b) == QCF_OK) check_sizes(who, c, b, Hq);
  return 0;
}

qcf_status qcf_paged_chunk_attn(const qcf_paged_kv* cache, const qcf_paged_batch* batch, const void* q, int64_t q_stride, int Hq,
                                float scale, int window, void* o, float* lse, void* ws, size_t ws_bytes, void* stream) {
  const char* who = "qcf_paged_chunk_attn";
  PagedView c;
  BatchView b;
  qcf_status s = check_paged(who, cache, batch, &c, &b);
  if (s == QCF_OK) s = check_sizes(who, c, b, Hq);
  if (s == QCF_OK) s = check_chunk(who, c, q, q_stride, Hq, scale, window, o, ws);
  if (s != QCF_OK) return s;
  if (b.n_seq == 0 || b.n_rows == 0) return QCF_OK;
  const ChunkArgs p{attn_args(q, q_stride, o, lse, Hq, c.Hkv, scale), cache->k, cache->v, 0, c.D, window};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = cache->dtype == QCF_BF16 ? chunk_launch<__nv_bfloat16, true>(c, b, p, st) : chunk_launch<__half, true>(c, b, p, st);
  return e == cudaSuccess ? QCF_OK : cuda_error(e, "qcf_paged_chunk_attn: launch");
}

}  // extern "C"
