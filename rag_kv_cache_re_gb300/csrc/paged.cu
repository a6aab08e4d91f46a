// New keys and values of a batch of sequences written into their cache pages, the position
// rotation applied on the way, and the queries of the same rows rotated in the same launch.
#include <algorithm>

#include "paged.cuh"

namespace qcf {

qcf_status check_paged(const char* who, const qcf_paged_kv* c, const qcf_paged_batch* b, PagedView* cv, BatchView* bv) {
  if (!c || !b || !c->k || !c->v || !b->row_start || !b->kv_len || !b->page_table)
    return set_error(QCF_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (c->dtype != QCF_BF16 && c->dtype != QCF_F16) return set_error(QCF_ERR_INVALID_ARG, "%s: cache dtype %d", who, c->dtype);
  if (c->n_pages <= 0 || c->page_size < 8 || c->page_size > 256 || (c->page_size & (c->page_size - 1)))
    return set_error(QCF_ERR_SHAPE, "%s: %d pages of %d rows (a power of two, 8 to 256)", who, c->n_pages, c->page_size);
  if (c->Hkv <= 0 || c->Hkv > 65535 || (c->D != 16 && c->D != 64 && c->D != 128))
    return set_error(QCF_ERR_SHAPE, "%s: Hkv=%d D=%d", who, c->Hkv, c->D);
  if (c->row_stride < c->D || c->head_stride < c->D || c->page_stride < c->D)
    return set_error(QCF_ERR_SHAPE, "%s: cache strides below the head dim", who);
  if (c->page_stride % 8 || c->row_stride % 8 || c->head_stride % 8 || !aligned16(c->k) || !aligned16(c->v))
    return set_error(QCF_ERR_ALIGN, "%s: cache pointers and strides must be multiples of 16 bytes", who);
  if (b->n_seq < 0 || b->n_seq > 65535 || b->n_rows < 0 || b->max_q < 0 || b->max_len < 0 || b->table_stride <= 0 ||
      b->prefix_len < 0)
    return set_error(QCF_ERR_SHAPE, "%s: n_seq=%d n_rows=%d max_q=%d max_len=%d table_stride=%d prefix_len=%d", who, b->n_seq,
                     b->n_rows, b->max_q, b->max_len, b->table_stride, b->prefix_len);
  if (b->max_len > static_cast<int64_t>(b->table_stride) * c->page_size)
    return set_error(QCF_ERR_SHAPE, "%s: max_len=%d exceeds %d pages of %d rows", who, b->max_len, b->table_stride, c->page_size);
  if (static_cast<int64_t>(b->prefix_len) + b->max_len > INT32_MAX - 512)
    return set_error(QCF_ERR_SHAPE, "%s: prefix_len + max_len exceed 31 bits", who);
  if (b->prefix_len > 0 && !b->prefix_pages) return set_error(QCF_ERR_INVALID_ARG, "%s: prefix_pages is NULL", who);
  cv->n_pages = c->n_pages;
  cv->page_shift = 0;
  while ((1 << cv->page_shift) < c->page_size) ++cv->page_shift;
  cv->Hkv = c->Hkv;
  cv->D = c->D;
  cv->page_stride = c->page_stride;
  cv->row_stride = c->row_stride;
  cv->head_stride = c->head_stride;
  *bv = BatchView{b->n_seq,  b->n_rows,     b->max_q,        b->max_len,    b->row_start,
                  b->kv_len, b->page_table, b->table_stride, b->prefix_len, b->prefix_pages};
  return QCF_OK;
}

struct AppendArgs {
  const void* k_new;
  const void* v_new;
  int64_t kv_stride;
  const void* q;
  int64_t q_stride;
  void* q_out;
  int64_t q_out_stride;
  int Hq;             // 0: no queries
  void* k;
  void* v;
  const float* cos_t;
  const float* sin_t;
  int max_pos, R;     // R = 0: nothing is rotated
  int interleaved;
};

// A CTA takes `rows` rows and `chunks` of their chunks of 4 heads (queries, keys, values in turn),
// one thread per (row, chunk, item): every load is issued before the first warps know where their
// rows go (one warp per row looks up the sequence, the position and the page).  V: pairs per item
// (see item_at).  HBM-bound for many rows, 737 MB in 117 us (6.3 TB/s; 177 us with the lookup
// before the loads), and by that chain of lookups for few: 61 MB of 64 short sequences in 16 us,
// 16 rows in 3.9.  Four CTAs an SM leave 64 registers: pairs of neighbours spill 8 bytes a thread,
// halves 92, which costs nothing (the 737 MB with halves: 114 us).
constexpr int kAppendThreads = 256;
constexpr int kAppendHeads = 4;

template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kAppendThreads, 4) paged_append_kernel(const PagedView c, const BatchView b, const AppendArgs p,
                                                                      int rows, int chunks, unsigned int* status) {
  __shared__ int64_t slot_s[kAppendThreads / 32];   // the row's place in the cache, -1: nowhere
  __shared__ int pos_s[kAppendThreads / 32];        // the row's position, -1: not a row of the batch
  const int items = c.D / 2 / V;
  const int unit = threadIdx.x / items, item = threadIdx.x - unit * items;
  const int r = unit / chunks;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * rows + r;
  int chunk = blockIdx.y * chunks + unit - r * chunks;
  const int cq = (p.Hq + kAppendHeads - 1) / kAppendHeads, ck = (c.Hkv + kAppendHeads - 1) / kAppendHeads;
  const bool is_q = chunk < cq, is_v = chunk >= cq + ck;
  const bool real = r < rows && row < b.n_rows && chunk < cq + 2 * ck;
  const int h0 = (is_q ? chunk : is_v ? chunk - cq - ck : chunk - cq) * kAppendHeads, H = is_q ? p.Hq : c.Hkv;
  const ItemAt at = item_at<V, INTER>(item, is_v ? 0 : p.R);
  const T* src = is_q ? static_cast<const T*>(p.q) + row * p.q_stride
                      : (is_v ? static_cast<const T*>(p.v_new) : static_cast<const T*>(p.k_new)) + row * p.kv_stride;
  Run<T, V> x[kAppendHeads], y[kAppendHeads];
#pragma unroll
  for (int i = 0; i < kAppendHeads; ++i)
    if (real && h0 + i < H) {
      x[i].load(src + (h0 + i) * c.D + at.a);
      y[i].load(src + (h0 + i) * c.D + at.b);
    }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row_w = blockIdx.x * rows + warp;
  if (warp < rows && row_w < b.n_rows) {
    const int seq = warp_seq_of_row(b, row_w);
    int pos = -1;
    int64_t slot = -1;
    if (seq >= 0) {
      const SeqSpan s = seq_span(b, seq);
      const bool first = lane == 0 && blockIdx.y == 0;
      if (s.bad) {
        if (first) flag_status(status, QCF_DEV_BAD_INDEX);
      } else if (row_w < s.row0 + s.nq) {
        const int own = s.len - s.nq + (row_w - s.row0);
        pos = b.prefix_len + own;
        slot = slot_of(c, b.page_table + static_cast<int64_t>(seq) * b.table_stride, own);
        if (p.R && pos >= p.max_pos) pos = slot = -1;
        if (slot < 0 && first) flag_status(status, QCF_DEV_BAD_INDEX);
      }
    }
    if (lane == 0) {
      pos_s[warp] = pos;
      slot_s[warp] = slot;
    }
  }
  __syncthreads();
  if (!real) return;
  const int pos = pos_s[r];
  const int64_t slot = slot_s[r];
  if (pos < 0 || (!is_q && slot < 0)) return;
  if (at.turns) {
    const Angles<V> g = load_angles<V>(p.cos_t, p.sin_t, pos, p.R, item, false);
#pragma unroll
    for (int i = 0; i < kAppendHeads; ++i)
      if (h0 + i < H) turn_item<T, V, INTER>(x[i], y[i], g);
  }
  T* dst = is_q ? static_cast<T*>(p.q_out) + row * p.q_out_stride : (is_v ? static_cast<T*>(p.v) : static_cast<T*>(p.k)) + slot;
  const int64_t step = is_q ? c.D : c.head_stride;
#pragma unroll
  for (int i = 0; i < kAppendHeads; ++i)
    if (h0 + i < H) {
      x[i].store(dst + (h0 + i) * step + at.a);
      y[i].store(dst + (h0 + i) * step + at.b);
    }
}

template <typename T, int V>
static cudaError_t append_launch(const PagedView& c, const BatchView& b, const AppendArgs& a, cudaStream_t st) {
  const int items = c.D / 2 / V;
  const int all = (a.Hq + kAppendHeads - 1) / kAppendHeads + 2 * ((c.Hkv + kAppendHeads - 1) / kAppendHeads);
  const int chunks = std::min(all, kAppendThreads / items);
  const int rows = std::min({kAppendThreads / (items * chunks), kAppendThreads / 32, b.n_rows});
  const int threads = (std::max(rows * 32, rows * chunks * items) + 31) / 32 * 32;
  LaunchScope ls(KC_APPEND, st);
  const auto kernel = a.interleaved ? paged_append_kernel<T, V, true> : paged_append_kernel<T, V, false>;
  kernel<<<dim3((b.n_rows + rows - 1) / rows, (all + chunks - 1) / chunks), threads, 0, st>>>(
      c, b, a, rows, chunks, device_status_ptr());
  return cudaGetLastError();
}

template <typename T>
static cudaError_t append_type(const PagedView& c, const BatchView& b, const AppendArgs& a, cudaStream_t st) {
  switch (a.R ? item_width(a.R, c.D) : 8) {
    case 8: return append_launch<T, 8>(c, b, a, st);
    case 4: return append_launch<T, 4>(c, b, a, st);
    case 2: return append_launch<T, 2>(c, b, a, st);
    default: return append_launch<T, 1>(c, b, a, st);
  }
}

}  // namespace qcf

using namespace qcf;

extern "C" {

qcf_status qcf_paged_append(const qcf_paged_kv* cache, const qcf_paged_batch* batch, const void* k_new, const void* v_new,
                            int64_t kv_stride, const qcf_rope_table* t, int mode, const void* q, int64_t q_stride, void* q_out,
                            int64_t q_out_stride, int Hq, void* stream) {
  const char* who = "qcf_paged_append";
  PagedView c;
  BatchView b;
  const qcf_status s = check_paged(who, cache, batch, &c, &b);
  if (s != QCF_OK) return s;
  if (!k_new || !v_new || (q == nullptr) != (q_out == nullptr) || (t && (!t->cos || !t->sin)))
    return set_error(QCF_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (mode & ~QCF_ROPE_INTERLEAVED) return set_error(QCF_ERR_INVALID_ARG, "%s: mode=%d", who, mode);
  if (t && (t->head_dim < 2 || (t->head_dim & 1) || t->head_dim > c.D || t->max_pos <= 0))
    return set_error(QCF_ERR_SHAPE, "%s: rotated width %d of head dim %d", who, t->head_dim, c.D);
  if (q && (Hq <= 0 || Hq > 65535)) return set_error(QCF_ERR_SHAPE, "%s: Hq=%d", who, Hq);
  if (kv_stride < static_cast<int64_t>(c.Hkv) * c.D ||
      (q && (q_stride < static_cast<int64_t>(Hq) * c.D || q_out_stride < static_cast<int64_t>(Hq) * c.D ||
             (q == q_out && q_stride != q_out_stride))))
    return set_error(QCF_ERR_SHAPE, "%s: row strides %lld, %lld, %lld are too short", who, (long long)kv_stride,
                     (long long)q_stride, (long long)q_out_stride);
  if (take_fault(4) || !aligned16(k_new) || !aligned16(v_new) || kv_stride % 8 ||
      (q && (!aligned16(q) || !aligned16(q_out) || q_stride % 8 || q_out_stride % 8)) ||
      (t && (!aligned16(t->cos) || !aligned16(t->sin))))
    return set_error(QCF_ERR_ALIGN, "%s: pointers and row strides must be multiples of 16 bytes", who);
  if (take_fault(1)) return set_error(QCF_ERR_INVALID_ARG, "%s: injected invalid index table", who);
  if (b.n_seq == 0 || b.n_rows == 0) return QCF_OK;
  const AppendArgs a{k_new, v_new,    kv_stride, q,
                     q_stride, q_out, q_out_stride, q ? Hq : 0,
                     cache->k, cache->v, t ? t->cos : nullptr, t ? t->sin : nullptr,
                     t ? t->max_pos : 0, t ? t->head_dim : 0, mode & QCF_ROPE_INTERLEAVED};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = cache->dtype == QCF_BF16 ? append_type<__nv_bfloat16>(c, b, a, st) : append_type<__half>(c, b, a, st);
  return e == cudaSuccess ? QCF_OK : cuda_error(e, "qcf_paged_append: launch");
}

}  // extern "C"
