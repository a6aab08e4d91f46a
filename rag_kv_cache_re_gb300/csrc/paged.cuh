// The paged cache and batch descriptors as kernels see them, and the lookups they share.
#pragma once

#include "rotary.cuh"

namespace qcf {

struct PagedView {
  int n_pages, page_shift, Hkv, D;
  int64_t page_stride, row_stride, head_stride;   // entries
};

struct BatchView {
  int n_seq, n_rows, max_q, max_len;
  const int32_t* row_start;
  const int32_t* kv_len;
  const int32_t* page_table;
  int table_stride, prefix_len;
  const int32_t* prefix_pages;
};

// A sequence's share of the batch; nq = 0 when the sequence has no rows or breaks a bound.
struct SeqSpan {
  int row0, nq, len;
  bool bad;
};
__device__ __forceinline__ SeqSpan seq_span(const BatchView& b, int seq) {
  SeqSpan s;
  s.row0 = b.row_start[seq];
  const int end = b.row_start[seq + 1];
  s.len = b.kv_len[seq];
  s.bad = s.row0 < 0 || end < s.row0 || end > b.n_rows || end - s.row0 > b.max_q || s.len < end - s.row0 || s.len > b.max_len;
  s.nq = s.bad ? 0 : end - s.row0;
  return s;
}

// The sequence of a row: the last one whose row_start is at most `row`, or -1 before the first.
// All 32 lanes of a warp call it with the same row; each round narrows the range by 32.
__device__ __forceinline__ int warp_seq_of_row(const BatchView& b, int row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = b.n_seq;   // the answer + 1 lies in [lo, lo + n]
  while (n > 0) {
    const int step = (n + 31) / 32;
    // lane i looks at the last entry of its piece [lo + i step, lo + (i + 1) step)
    const int i = min(lane * step + step, n) - 1;
    const bool le = b.row_start[lo + i] <= row;
    const int pieces = __popc(__ballot_sync(0xffffffffu, le && lane * step < n));
    const int skip = min(pieces * step, n);
    lo += skip;
    n = step > 1 ? min(step, n - skip) : 0;
    if (n > 0) --n;   // the last entry of the next piece is above `row`
  }
  return lo - 1;
}

// Base entry of own token `p` of a sequence (its page's row, head 0), or -1 for a page outside the cache.
__device__ __forceinline__ int64_t slot_of(const PagedView& c, const int32_t* __restrict__ pages, int p) {
  const int page = pages[p >> c.page_shift];
  if (page < 0 || page >= c.n_pages) return -1;
  return page * c.page_stride + (p & ((1 << c.page_shift) - 1)) * c.row_stride;
}

// Host checks shared by the entry points (paged.cu).
qcf_status check_paged(const char* who, const qcf_paged_kv* c, const qcf_paged_batch* b, PagedView* cv, BatchView* bv);

}  // namespace qcf
