// The pages of a cache as sequences come, branch, grow, end: reference counts, page tables and lengths on the
// device, the same page ids in every layer.
//
// Each call is two kernels.  The plan, one CTA, reads counts, tables and lengths, takes the pages it
// needs (always the lowest ids free before the call, in the order of its arguments) and leaves what is
// to be done in the scratch; it decides for the whole call, so that a bad argument or a lack of pages
// changes nothing.  The apply kernel writes tables, counts and lengths from it and copies rows of pages in all layers.
#include <algorithm>

#include "paged.cuh"

namespace qcf {

constexpr int kMaxCaches = 256;
constexpr int kPlanThreads = 1024;
constexpr int kApplyThreads = 256;

struct PoolView {
  int n_pages, page_shift, n_seq, table_stride, n;   // n: arguments of the call
  int32_t* refs;
  int32_t* table;
  int32_t* kv_len;
};

// One argument's share of the plan.
struct PlanItem {
  int seq, from;        // sequence written, sequence read (fork)
  int keep;             // pages that stay (resize), full pages shared (fork)
  int drop0, drop1;     // columns whose pages are given back
  int add0, add1;       // columns that get new pages, first .. of the list
  int first;
  int len;              // length after the call
  int copy_col;         // the column of a page held in part that is copied to the first new one; -1: none
  int copy_src, copy_rows;
};
struct PlanHead {
  int ok, copies, live, unused;
};
struct PlanView {
  PlanHead* head;
  PlanItem* items;
  int32_t* list;    // pages taken; compact: places that pages move to
  int32_t* list2;   // compact: pages that move
  int32_t* map;     // compact: new id of a page at or above the live count
};

struct CachePtrs {
  void* p[2 * kMaxCaches];
};
struct CopyShape {
  int n_ptrs, Hkv, page_size;
  int d_shift;                                    // log2 of a head's 16-byte pieces
  int64_t page_stride, row_stride, head_stride;   // 16-byte pieces
  bool rows_outer, dense;                         // [row][head] or [head][row]; a page has no gaps
};

// Sum of v over the threads before this one, and over the block.  met: 32 entries, of its own for calls that follow
// each other without a barrier between (every warp adds the warps' sums for itself, which saves two).
template <typename I>
__device__ __forceinline__ I block_scan(I v, I* met, I* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  I run = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const I u = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += u;
  }
  if (lane == 31) met[warp] = run;
  __syncthreads();
  I w = met[lane];
  const I own = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const I u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += u;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  return run - v + __shfl_sync(0xffffffffu, w - own, warp);
}

// A pass over the counts: a warp has N x 32 ids in a row, a lane every 32nd of them, so that loads and lists are coalesced
// and ranks are votes.
template <int N>
__device__ __forceinline__ int64_t id_at(int64_t base, int e) { return base + (threadIdx.x >> 5) * (32 * N) + e * 32 + (threadIdx.x & 31); }
// The counts of this lane's ids; -1 behind the end.
template <int N>
__device__ __forceinline__ void load_refs(const PoolView& p, int64_t base, int* r) {
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const int64_t id = id_at<N>(base, e);
    r[e] = id < p.n_pages ? p.refs[id] : -1;
  }
}

// The lowest `want` free ids, ascending, into list; how many there are, at most want.  r: the counts of the first pass.  Free
// pages are mostly found early: short passes, the next one's counts on their way.
constexpr int kFreeIds = 4;
__device__ int take_free(const PoolView& p, int want, int32_t* list, int* met, int* r) {
  const unsigned below = (1u << (threadIdx.x & 31)) - 1u;
  int found = 0;
  for (int64_t base = 0; base < p.n_pages && found < want; base += kPlanThreads * kFreeIds) {
    int next[kFreeIds];
    load_refs<kFreeIds>(p, base + kPlanThreads * kFreeIds, next);
    int n = 0, total;
#pragma unroll
    for (int e = 0; e < kFreeIds; ++e) n += __popc(__ballot_sync(0xffffffffu, r[e] == 0));
    // a warp's count once, in its last lane
    int at = found + __shfl_sync(0xffffffffu, block_scan((threadIdx.x & 31) == 31 ? n : 0, met, &total), 31);
#pragma unroll
    for (int e = 0; e < kFreeIds; ++e) {
      const unsigned free = __ballot_sync(0xffffffffu, r[e] == 0);
      const int place = at + __popc(free & below);
      if (r[e] == 0 && place < want) list[place] = static_cast<int>(id_at<kFreeIds>(base, e));
      at += __popc(free);
      r[e] = next[e];
    }
    found += total;
    __syncthreads();   // met may be written again
  }
  return min(found, want);
}

__device__ __forceinline__ int pages_of(const PoolView& p, int len) { return (len + (1 << p.page_shift) - 1) >> p.page_shift; }

// Marks sequence b in the bit set; whether it was marked before.
__device__ __forceinline__ bool mark(unsigned* set, int b) { return atomicOr(&set[b >> 5], 1u << (b & 31)) >> (b & 31) & 1u; }

// FORK: a = sources, b = destinations.  Otherwise (resize): a = sequences (NULL: 0, 1, ..), b = new lengths.
// Bound by the chain of loads an argument takes (itself, its sequence's length, the table, the count of a page): 2 us, beside 2 of
// the launch.
template <bool FORK>
__global__ void __launch_bounds__(kPlanThreads) pages_plan_kernel(const PoolView p, const int32_t* a, const int32_t* b, const PlanView out,
                                                                  unsigned int* status) {
  __shared__ int64_t sums[32];
  __shared__ int met[32];
  __shared__ unsigned named[2048];
  const int words = (p.n_seq + 31) / 32, most = p.table_stride << p.page_shift;
  for (int i = threadIdx.x; i < words; i += kPlanThreads) named[i] = 0;
  pdl_wait();
  pdl_launch_dependents();   // what applies the plan comes up meanwhile (turnover 11.3 -> 10.9 us)
  __syncthreads();
  bool bad = false;
  PlanItem mine = {};   // of the first 1024 arguments, which are mostly all
  auto read = [&](int i, PlanItem& it) {
    it.seq = FORK ? b[i] : a ? a[i] : i;
    it.from = FORK ? a[i] : it.seq;
    it.copy_col = -1;
    const int to = FORK ? 0 : b[i];
    if (it.seq < 0 || it.seq >= p.n_seq || it.from < 0 || it.from >= p.n_seq || to < 0 || to > most) return false;
    const int now = p.kv_len[it.seq], src = p.kv_len[it.from];
    if (mark(named, it.seq) || now < 0 || now > most || src < 0 || src > most) return false;   // each sequence is written once
    const int kept = FORK ? src : min(now, to), part = kept & ((1 << p.page_shift) - 1);
    it.len = FORK ? src : to;
    it.keep = kept >> p.page_shift;
    if (part > 0 && (FORK || now != to)) {
      // a page held in part is copied: by fork always, by resize where others hold it too
      const int page = p.table[static_cast<int64_t>(it.from) * p.table_stride + it.keep];
      if (page < 0 || page >= p.n_pages) return false;
      if (FORK || p.refs[page] > 1) {
        it.copy_src = page;
        it.copy_col = it.keep;
        it.copy_rows = part;
      }
    }
    it.drop1 = pages_of(p, now);
    it.drop0 = FORK ? 0 : min(pages_of(p, to), it.drop1);
    it.add0 = FORK ? 0 : it.drop1;
    it.add1 = FORK ? 0 : max(pages_of(p, to), it.drop1);
    return true;
  };
  for (int i = threadIdx.x; i < p.n; i += kPlanThreads) {
    PlanItem it = {};
    bad |= !read(i, it);
    if (i == threadIdx.x) mine = it; else out.items[i] = it;
  }
  int r[kFreeIds];
  load_refs<kFreeIds>(p, 0, r);   // on their way under the sums
  bad = __syncthreads_or(bad);
  int wanted = 0, copies = 0;
  for (int i0 = 0; i0 < p.n && !bad; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    PlanItem it = {};
    if (i < p.n) it = i0 == 0 ? mine : out.items[i];
    const bool copied = i < p.n && it.copy_col >= 0;
    const bool wrong = FORK && i < p.n && (named[it.from >> 5] >> (it.from & 31) & 1u);   // a source that is written
    const int take = i < p.n ? (copied ? 1 : 0) + it.add1 - it.add0 : 0;
    // new pages, and above them copies and wrong arguments, in one sum
    int64_t total;
    const int64_t before = block_scan(take | static_cast<int64_t>(copied) << 32 | static_cast<int64_t>(wrong) << 48, sums, &total);
    it.first = wanted + static_cast<int>(before & 0xffffffff);
    wanted = static_cast<int>(min(wanted + (total & 0xffffffff), static_cast<int64_t>(p.n_pages) + 1));
    copies += static_cast<int>(total >> 32 & 0xffff);
    bad |= total >> 48 != 0;
    if (i < p.n) out.items[i] = it;
    if (i0 + kPlanThreads < p.n) __syncthreads();   // sums may be written again
  }
  const bool over = wanted > p.n_pages;
  const int found = bad || over ? 0 : take_free(p, wanted, out.list, met, r);
  if (threadIdx.x == 0) {
    const bool few = !bad && (over || found < wanted);
    if (bad) flag_status(status, QCF_DEV_BAD_INDEX);
    if (few) flag_status(status, QCF_DEV_NO_PAGES);
    *out.head = PlanHead{!bad && !few, copies, 0, 0};
  }
}

constexpr int kCompactIds = 16, kCompactPass = kPlanThreads * kCompactIds;
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const PoolView p, const PlanView out, int32_t* n_live,
                                                                    unsigned int* status) {
  __shared__ int64_t met[2][32];
  const unsigned below = (1u << (threadIdx.x & 31)) - 1u;
  const bool last = (threadIdx.x & 31) == 31;
  int r[kCompactIds];
  int64_t total;
  int count = 0;
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t base = 0; base < p.n_pages; base += kCompactPass) {
    load_refs<kCompactIds>(p, base, r);
#pragma unroll
    for (int e = 0; e < kCompactIds; ++e) count += r[e] > 0;
  }
  const int most = p.table_stride << p.page_shift;
  bool bad = false;
  for (int i = threadIdx.x; i < p.n_seq; i += kPlanThreads) {
    const int len = p.kv_len[i];
    bad |= len < 0 || len > most;
  }
  block_scan(count | static_cast<int64_t>(bad) << 32, met[0], &total);
  bad = total >> 32 != 0;
  const int live = static_cast<int>(total & 0xffffffff);
  int holes = 0, moves = 0;   // below `live` there are as many free pages as live ones above
  for (int64_t base = 0; base < p.n_pages; base += kCompactPass) {
    if (p.n_pages > kCompactPass) load_refs<kCompactIds>(p, base, r);   // one pass has them still
    int h = 0, m = 0;
#pragma unroll
    for (int e = 0; e < kCompactIds; ++e) {
      const int64_t id = id_at<kCompactIds>(base, e);
      h += __popc(__ballot_sync(0xffffffffu, id < live && r[e] <= 0));
      m += __popc(__ballot_sync(0xffffffffu, id >= live && r[e] > 0));
    }
    const int64_t before = __shfl_sync(0xffffffffu, block_scan(last ? h | static_cast<int64_t>(m) << 32 : 0, met[1], &total), 31);
    int ha = holes + static_cast<int>(before & 0xffffffff), ma = moves + static_cast<int>(before >> 32);
#pragma unroll
    for (int e = 0; e < kCompactIds; ++e) {
      const int64_t id = id_at<kCompactIds>(base, e);
      const bool hole = id < live && r[e] <= 0, move = id >= live && r[e] > 0;   // -1 behind the last page: neither
      const unsigned hs = __ballot_sync(0xffffffffu, hole), ms = __ballot_sync(0xffffffffu, move);
      if (hole) out.list[ha + __popc(hs & below)] = static_cast<int>(id);
      if (move) out.list2[ma + __popc(ms & below)] = static_cast<int>(id);
      if (id >= live && id < p.n_pages) out.map[id] = move ? ma + __popc(ms & below) : -1;
      ha += __popc(hs);
      ma += __popc(ms);
    }
    holes += static_cast<int>(total & 0xffffffff);
    moves += static_cast<int>(total >> 32);
    __syncthreads();   // met may be written again
  }
  if (threadIdx.x == 0) {
    if (bad) flag_status(status, QCF_DEV_BAD_INDEX);
    *out.head = PlanHead{!bad, moves, live, 0};
    *n_live = bad ? -1 : live;   // nothing moves: no count may say which pages are free
  }
}

// Copies the first rows of pages to others in every layer, keys and values.  A CTA takes 16 KB of one tensor's
// page at a time; what the next one copies is looked up under the loads of this one.  Bound by HBM: 1422 MB read and written as
// a cache is compacted in 212 to 216 us (6.6 TB/s), the call 230.
constexpr int kCopyPieces = 1024;   // 16-byte pieces of a CTA's part
struct CopyItem {
  int src, dst, rows;   // rows 0: nothing
};
template <typename F>
__device__ __forceinline__ void copy_pages(const CopyShape& s, const CachePtrs& c, int parts, int n, F item) {
  const unsigned per_item = s.n_ptrs * parts;
  const int per_row = s.Hkv << s.d_shift;
  constexpr int N = kCopyPieces / kApplyThreads;
  unsigned i = blockIdx.x / per_item, rest = blockIdx.x - i * per_item;   // item, and which part of which tensor
  if (i >= static_cast<unsigned>(n)) return;
  CopyItem it = item(static_cast<int>(i));
  while (true) {
    const unsigned ptr = rest / parts, part = rest - ptr * parts;
    const uint4* from = static_cast<const uint4*>(c.p[ptr]) + it.src * s.page_stride;
    uint4* to = static_cast<uint4*>(c.p[ptr]) + it.dst * s.page_stride;
    const int rows = it.rows, end = min(rows * per_row, static_cast<int>(part + 1) * kCopyPieces);
    const bool dense = s.dense && (s.rows_outer || rows == s.page_size);
    uint4 v[N];
    int64_t at[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int e = part * kCopyPieces + j * kApplyThreads + threadIdx.x;
      if (e < end) {
        if (dense) {
          at[j] = e;
        } else if (s.rows_outer) {
          const int row = e / per_row, x = e - row * per_row;
          at[j] = row * s.row_stride + (x >> s.d_shift) * s.head_stride + (x & ((1 << s.d_shift) - 1));
        } else {
          const int per_head = rows << s.d_shift, head = e / per_head, x = e - head * per_head;
          at[j] = head * s.head_stride + (x >> s.d_shift) * s.row_stride + (x & ((1 << s.d_shift) - 1));
        }
        v[j] = __ldcs(from + at[j]);
      }
    }
    rest += gridDim.x;
    i += rest / per_item;
    rest %= per_item;
    const bool more = i < static_cast<unsigned>(n);
    if (more) it = item(static_cast<int>(i));
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (part * kCopyPieces + j * kApplyThreads + threadIdx.x < static_cast<unsigned>(end)) __stcs(to + at[j], v[j]);
    if (!more) return;
  }
}

__device__ __forceinline__ void add_ref(const PoolView& p, int page, int by, unsigned int* status) {
  if (page >= 0 && page < p.n_pages)
    atomicAdd(&p.refs[page], by);
  else
    flag_status(status, QCF_DEV_BAD_INDEX);
}

template <bool FORK>
__global__ void __launch_bounds__(kApplyThreads) pages_apply_kernel(const PoolView p, const PlanView plan, const CopyShape s,
                                                                    const __grid_constant__ CachePtrs c, int parts, unsigned int* status) {
  pdl_wait();
  const PlanHead head = *plan.head;
  if (!head.ok) return;
  for (int i = blockIdx.x; i < p.n; i += gridDim.x) {
    const PlanItem it = plan.items[i];
    int32_t* row = p.table + static_cast<int64_t>(it.seq) * p.table_stride;
    const int32_t* from = p.table + static_cast<int64_t>(it.from) * p.table_stride;
    const int split = it.copy_col >= 0 ? 1 : 0;
    const int end = max(max(it.drop1, it.add1), it.keep + split);
    for (int col = threadIdx.x; col < end; col += kApplyThreads) {
      const int old = row[col];
      int now = old;
      if (col == it.copy_col)
        now = plan.list[it.first];
      else if (FORK && col < it.keep)
        now = from[col];
      else if (col >= it.add0 && col < it.add1)
        now = plan.list[it.first + split + col - it.add0];
      if (FORK ? col < it.drop1 : (col >= it.drop0 && col < it.drop1) || col == it.copy_col) add_ref(p, old, -1, status);
      if (FORK ? col < it.keep + split : (col >= it.add0 && col < it.add1) || col == it.copy_col) add_ref(p, now, 1, status);
      if (now != old) row[col] = now;
    }
    if (threadIdx.x == 0) p.kv_len[it.seq] = it.len;
  }
  if (head.copies == 0) return;
  copy_pages(s, c, parts, p.n, [&](int i) {
    const PlanItem it = plan.items[i];
    return it.copy_col < 0 ? CopyItem{0, 0, 0} : CopyItem{it.copy_src, plan.list[it.first], it.copy_rows};
  });
}

__global__ void __launch_bounds__(kApplyThreads) compact_apply_kernel(const PoolView p, const PlanView plan, const CopyShape s,
                                                                      const __grid_constant__ CachePtrs c, int parts, unsigned int* status) {
  pdl_wait();
  const PlanHead head = *plan.head;
  if (!head.ok || head.copies == 0) return;
  for (int seq = blockIdx.x; seq < p.n_seq; seq += gridDim.x) {
    int32_t* row = p.table + static_cast<int64_t>(seq) * p.table_stride;
    const int held = pages_of(p, p.kv_len[seq]);
    for (int col = threadIdx.x; col < held; col += kApplyThreads) {
      const int old = row[col];
      if (old >= 0 && old < head.live) continue;
      const int now = old < 0 || old >= p.n_pages ? -1 : plan.map[old];
      if (now >= 0)
        row[col] = plan.list[now];
      else
        flag_status(status, QCF_DEV_BAD_INDEX);   // outside the cache, or not counted: left as it is
    }
  }
  for (int64_t m = static_cast<int64_t>(blockIdx.x) * kApplyThreads + threadIdx.x; m < head.copies; m += static_cast<int64_t>(gridDim.x) * kApplyThreads) {
    p.refs[plan.list[m]] = p.refs[plan.list2[m]];
    p.refs[plan.list2[m]] = 0;
  }
  copy_pages(s, c, parts, head.copies, [&](int m) { return CopyItem{plan.list2[m], plan.list[m], s.page_size}; });
}

// ------------------------------------------------------------------ host

static qcf_status check_pool(const char* who, const qcf_page_pool* pool, int n, PoolView* v, CopyShape* s, CachePtrs* c) {
  if (!pool || !pool->caches || !pool->refs || (pool->n_seq > 0 && (!pool->page_table || !pool->kv_len)))
    return set_error(QCF_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (pool->n_caches < 1 || pool->n_caches > kMaxCaches || pool->n_seq < 0 || pool->n_seq > 65535 || pool->table_stride <= 0 ||
      pool->table_stride > 1 << 20 || n < 0 || n > pool->n_seq)
    return set_error(QCF_ERR_SHAPE, "%s: n_caches=%d n_seq=%d table_stride=%d n=%d", who, pool->n_caches, pool->n_seq, pool->table_stride, n);
  const qcf_paged_kv& first = pool->caches[0];
  // the checks of a cache, with a batch that has no sequences
  qcf_paged_batch none = {};
  none.row_start = none.kv_len = none.page_table = pool->refs;   // only looked at for NULL
  none.table_stride = 1;
  PagedView pv;
  BatchView bv;
  for (int i = 0; i < pool->n_caches; ++i) {
    const qcf_paged_kv& k = pool->caches[i];
    const qcf_status st = check_paged(who, &k, &none, &pv, &bv);
    if (st != QCF_OK) return st;
    if (k.dtype != first.dtype || k.n_pages != first.n_pages || k.page_size != first.page_size || k.Hkv != first.Hkv || k.D != first.D ||
        k.page_stride != first.page_stride || k.row_stride != first.row_stride || k.head_stride != first.head_stride)
      return set_error(QCF_ERR_SHAPE, "%s: cache %d has another layout than the first", who, i);
    c->p[2 * i] = k.k;
    c->p[2 * i + 1] = k.v;
  }
  if (!aligned16(pool->refs) || (reinterpret_cast<uintptr_t>(pool->page_table) & 3u) || (reinterpret_cast<uintptr_t>(pool->kv_len) & 3u))
    return set_error(QCF_ERR_ALIGN, "%s: refs must be a multiple of 16 bytes, page_table and kv_len of 4", who);
  *v = PoolView{pv.n_pages, pv.page_shift, pool->n_seq, pool->table_stride, n, pool->refs, pool->page_table, pool->kv_len};
  s->n_ptrs = 2 * pool->n_caches;
  s->Hkv = pv.Hkv;
  s->page_size = first.page_size;
  s->d_shift = pv.D == 16 ? 1 : pv.D == 64 ? 3 : 4;
  s->page_stride = pv.page_stride / 8;
  s->row_stride = pv.row_stride / 8;
  s->head_stride = pv.head_stride / 8;
  s->rows_outer = pv.row_stride >= pv.head_stride;
  s->dense = s->rows_outer ? (pv.head_stride == pv.D || pv.Hkv == 1) && pv.row_stride == static_cast<int64_t>(pv.Hkv) * pv.D
                           : pv.row_stride == pv.D && pv.head_stride == static_cast<int64_t>(first.page_size) * pv.D;
  return QCF_OK;
}

static size_t plan_layout(const PoolView& p, void* base, PlanView* v) {
  uint8_t* at = static_cast<uint8_t*>(base);
  size_t used = 0;
  auto take = [&](size_t bytes) {
    uint8_t* r = at + used;
    used += align_up(bytes, 256);
    return r;
  };
  const size_t ids = static_cast<size_t>(p.n_pages) * sizeof(int32_t);
  v->head = reinterpret_cast<PlanHead*>(take(sizeof(PlanHead)));
  v->items = reinterpret_cast<PlanItem*>(take(static_cast<size_t>(p.n) * sizeof(PlanItem)));
  v->list = reinterpret_cast<int32_t*>(take(ids));
  v->list2 = reinterpret_cast<int32_t*>(take(ids));
  v->map = reinterpret_cast<int32_t*>(take(ids));
  return used;
}

struct PoolCall {
  PoolView p;
  CopyShape s;
  CachePtrs c;
  PlanView plan;
  int parts;
};

static qcf_status open_pool(const char* who, const qcf_page_pool* pool, int n, void* ws, size_t ws_bytes, PoolCall* k) {
  const qcf_status st = check_pool(who, pool, n, &k->p, &k->s, &k->c);
  if (st != QCF_OK) return st;
  if (take_fault(4) || (reinterpret_cast<uintptr_t>(ws) & 255u)) return set_error(QCF_ERR_ALIGN, "%s: ws must be a multiple of 256 bytes", who);
  if (take_fault(1)) return set_error(QCF_ERR_INVALID_ARG, "%s: injected invalid index table", who);
  const size_t need = plan_layout(k->p, ws, &k->plan);
  if (take_fault(2) || !ws || ws_bytes < need) return set_error(QCF_ERR_WORKSPACE, "%s: workspace %zu < %zu", who, ws_bytes, need);
  k->parts = ((k->s.page_size * k->s.Hkv << k->s.d_shift) + kCopyPieces - 1) / kCopyPieces;
  return QCF_OK;
}

template <bool FORK>
static qcf_status pages_launch(const char* who, const PoolCall& k, const int32_t* a, const int32_t* b, cudaStream_t st) {
  {
    LaunchScope ls(KC_PAGES, st);
    const cudaError_t e = launch_pdl(pages_plan_kernel<FORK>, dim3(1), dim3(kPlanThreads), 0, st, k.p, a, b, k.plan, device_status_ptr());
    if (e != cudaSuccess) return cuda_error(e, who);
  }
  LaunchScope ls(KC_PAGES, st);
  const int64_t work = static_cast<int64_t>(k.p.n) * k.s.n_ptrs * k.parts;   // a CTA for each sequence's table, and each part of a copy
  const cudaError_t e = launch_pdl(pages_apply_kernel<FORK>, dim3(static_cast<unsigned>(std::min<int64_t>(work, num_sms() * 8))), dim3(kApplyThreads), 0, st, k.p, k.plan, k.s, k.c, k.parts,
                                   device_status_ptr());
  return e == cudaSuccess ? QCF_OK : cuda_error(e, who);
}

}  // namespace qcf

using namespace qcf;

extern "C" {

size_t qcf_pages_workspace_size(const qcf_page_pool* pool, int n) {
  PoolCall k;
  if (check_pool("qcf_pages_workspace_size", pool, n, &k.p, &k.s, &k.c) != QCF_OK) return 0;
  return plan_layout(k.p, nullptr, &k.plan);
}

qcf_status qcf_pages_fork(const qcf_page_pool* pool, const int32_t* src, const int32_t* dst, int n, void* ws, size_t ws_bytes, void* stream) {
  PoolCall k;
  const qcf_status s = open_pool("qcf_pages_fork", pool, n, ws, ws_bytes, &k);
  if (s != QCF_OK) return s;
  if (!src || !dst) return set_error(QCF_ERR_INVALID_ARG, "qcf_pages_fork: NULL pointer");
  return n == 0 ? QCF_OK : pages_launch<true>("qcf_pages_fork: launch", k, src, dst, static_cast<cudaStream_t>(stream));
}

qcf_status qcf_pages_resize(const qcf_page_pool* pool, const int32_t* seqs, const int32_t* new_len, int n, void* ws, size_t ws_bytes,
                            void* stream) {
  PoolCall k;
  const qcf_status s = open_pool("qcf_pages_resize", pool, n, ws, ws_bytes, &k);
  if (s != QCF_OK) return s;
  if (!new_len) return set_error(QCF_ERR_INVALID_ARG, "qcf_pages_resize: NULL pointer");
  return n == 0 ? QCF_OK : pages_launch<false>("qcf_pages_resize: launch", k, seqs, new_len, static_cast<cudaStream_t>(stream));
}

qcf_status qcf_pages_compact(const qcf_page_pool* pool, int32_t* n_live, void* ws, size_t ws_bytes, void* stream) {
  PoolCall k;
  const qcf_status s = open_pool("qcf_pages_compact", pool, 0, ws, ws_bytes, &k);
  if (s != QCF_OK) return s;
  if (!n_live) return set_error(QCF_ERR_INVALID_ARG, "qcf_pages_compact: NULL pointer");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  {
    LaunchScope ls(KC_PAGES, st);
    const cudaError_t e = launch_pdl(compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, k.p, k.plan, n_live, device_status_ptr());
    if (e != cudaSuccess) return cuda_error(e, "qcf_pages_compact: launch");
  }
  LaunchScope ls(KC_PAGES, st);
  const cudaError_t e = launch_pdl(compact_apply_kernel, dim3(num_sms() * 8), dim3(kApplyThreads), 0, st, k.p, k.plan, k.s, k.c, k.parts,
                                   device_status_ptr());
  return e == cudaSuccess ? QCF_OK : cuda_error(e, "qcf_pages_compact: launch");
}

}  // extern "C"
