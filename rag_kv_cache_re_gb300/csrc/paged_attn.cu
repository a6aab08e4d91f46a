// Attention of a batch of sequences over a shared prefix and their own tokens, both in pages.
//
// With logits x_j = scale q.K_j, any set of keys P is summed up by M = max x_j, L = sum 2^(x_j - M)
// (x in powers of two) and O = sum 2^(x_j - M) V_j; two sets join by scaling each with
// 2^(M - max M).  The keys of a row are split into such parts: chunks of the prefix, scored for
// all rows of the batch together so that its K and V are read for many of them at once, and chunks of the sequence's
// own tokens.  A last kernel joins the parts of each row.
#include <algorithm>
#include <cmath>

#include "paged_attn.cuh"

namespace qcf {

constexpr int kMaxBatchSeqs = 2048;   // each CTA of the stream keeps 12 bytes of every sequence
constexpr int kMostTiles = INT32_MAX - (1 << 20);   // tiles of one call, with room for the shares' rounding

// ------------------------------------------------------------------ the stream, on warp tensor cores
//
// A unit is up to 16 score rows (new rows x the G query heads of one KV head; one m16 tile) of one
// sequence against its own keys, or 16 rows of the whole batch against the prefix.  The 32-key
// tiles of all units are dealt out evenly to persistent warps, whatever the lengths are, and every
// warp works alone: it keeps its own ring of K and V tiles full by tiled TMA (one box per page and
// 64 columns; pages behind a length, or outside the cache, read as zeros), ahead of the tile that it
// scores and across the borders of units, and no warp waits for another.  (Four warps that
// split a tile and met at two barriers took 1900 cycles per 64 keys of head dim 64, and 90 us for
// 386 MB of uneven sequences.)
// The maximum moves only when it grows by more than 2^8 (see kWeightLift), so most tiles rescale nothing.
// Bound by the K and V bytes; the rings keep 96 KB or more per SM in flight.  386 MB of uneven
// sequences of head dim 64 in 66 to 71 us (5.4 to 5.8 TB/s), 67 MB of short ones in 20, of which
// about 5 pass before the first tile is scored.  It serves any number of new rows, but a question of
// thousands of tokens is work for 128-row tiles (4 of 1024 rows: 622 us the call, 196 the floor).
template <int D>
struct StreamCfg {
  static constexpr int COLS = D < 64 ? D : 64, BOXES = D / COLS;
  static constexpr int BOX = kStreamKeys * COLS * 2;   // 32 keys x COLS entries
  static constexpr int TILE = BOXES * BOX;             // a K or V tile
  static constexpr int STAGES = D >= 64 ? 2 : 4;
  static constexpr int WARPS = D == 128 ? 6 : 12;      // 192 KB of rings (96 KB at head dim 16)
  static constexpr int RING = STAGES * 2 * TILE;       // of a warp
  static constexpr int FIXED = WARPS * (RING + STAGES * 8);
};
template <int D>
static size_t stream_smem(int n_seq) {
  return 1024 + StreamCfg<D>::FIXED + (3 * static_cast<size_t>(n_seq) + 3) * sizeof(int);
}

// Byte offset of 8 entries at column col of a key in a K or V tile, as TMA lays it out.
template <int D>
__device__ __forceinline__ uint32_t tile_at(int key, int col) {
  if constexpr (D >= 64)
    return static_cast<uint32_t>((col >> 6) * StreamCfg<D>::BOX) + sw128_off(key, (col & 63) >> 3);
  else
    return static_cast<uint32_t>(key * (D * 2) + col * 2);
}

__device__ __forceinline__ int stream_tiles_of(const SeqSpan& s, int G, int Hkv) {
  return s.nq == 0 ? 0 : (s.len + kStreamKeys - 1) / kStreamKeys * ((s.nq * G + kStreamRows - 1) / kStreamRows) * Hkv;
}

// What every CTA keeps of the batch in shared memory: small loads from global memory take 2 us once
// the rings are streaming, so nothing between two units may wait for one.
struct StreamDeal {
  const int* start;   // [n_seq + 2]: first tile of each sequence, the total, tiles to a worker
  const int* row0;    // [n_seq + 1]
  const int* len;     // [n_seq]
};

// One worker's share of one unit.
struct StreamSeg {
  bool pre;            // a unit of the prefix
  int g, rho0;         // KV head, first score row
  int row0, nq, len;   // of the sequence (the whole batch for the prefix)
  int t0, nt, tiles;   // key tiles of this share, of the unit
  int use;             // tiles of the share that any row of the unit sees (own tokens: the last ones none)
  int part;
  const int32_t* table;
};
// Walks a worker's share.  Only the first unit is found by division; every other begins at its first
// tile, behind the one before.
struct StreamWalk {
  int cur, end, seq, seq_end;   // tiles; the sequence and where it ends (the prefix: seq -1)
  StreamSeg at;
  __device__ void enter(const BatchView& b, const SharedPlan& p, const StreamDeal& deal) {   // the sequence that holds tile cur
    at.pre = seq < 0;
    if (at.pre) {
      at.row0 = 0;
      at.nq = b.n_rows;
      at.len = b.prefix_len;
      at.tiles = p.stream_tiles;
      at.table = b.prefix_pages;
      seq_end = deal.start[0];
    } else {
      at.row0 = deal.row0[seq];
      at.nq = deal.row0[seq + 1] - at.row0;
      at.len = deal.len[seq];
      at.tiles = (at.len + kStreamKeys - 1) / kStreamKeys;
      at.table = b.page_table + static_cast<int64_t>(seq) * b.table_stride;
      seq_end = deal.start[seq + 1];
    }
    at.g = at.rho0 = 0;
  }
  __device__ StreamWalk(const BatchView& b, const SharedPlan& p, const StreamDeal& deal, int worker, int Hkv) {
    const int* start = deal.start;
    const int total = start[b.n_seq], share = start[b.n_seq + 1];
    cur = static_cast<int>(min(static_cast<int64_t>(total), static_cast<int64_t>(worker) * share));
    end = min(total, cur + share);
    at.t0 = at.part = 0;
    if (cur >= end) return;
    int lo = -1, hi = b.n_seq;   // the last sequence that begins at or before cur (-1: the prefix), of those with tiles
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= cur) lo = mid; else hi = mid;
    }
    seq = lo;
    enter(b, p, deal);
    const int first = seq < 0 ? 0 : start[seq], u = (cur - first) / at.tiles;
    at.t0 = cur - first - u * at.tiles;
    at.g = u % Hkv;
    at.rho0 = u / Hkv * kStreamRows;
    if (at.t0 > 0) at.part = worker - (cur - at.t0) / share;
  }
  __device__ bool next(StreamSeg& s, const BatchView& b, const SharedPlan& p, const AttnArgs& a, const StreamDeal& deal, int Hkv) {
    if (cur >= end) return false;
    at.nt = min(at.tiles - at.t0, end - cur);
    const int reach =
        at.pre ? at.len : at.len - at.nq + min(at.nq, div_g(a, at.rho0 + kStreamRows - 1) + 1);   // keys any row sees
    at.use = max(0, min(at.nt, (reach + kStreamKeys - 1) / kStreamKeys - at.t0));
    s = at;
    cur += at.nt;
    at.t0 = at.part = 0;
    if (cur < end) {
      if (cur < seq_end) {
        if (++at.g == Hkv) {
          at.g = 0;
          at.rho0 += kStreamRows;
        }
      } else {
        do ++seq;
        while (deal.start[seq + 1] <= cur);
        enter(b, p, deal);
      }
    }
    return true;
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(StreamCfg<D>::WARPS * 32, 1)
    stream_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const PagedView c,
                       const BatchView b, const AttnArgs a, const SharedPlan p, const Workspace ws, unsigned int* status) {
  using Cfg = StreamCfg<D>;
  constexpr int ST = Cfg::STAGES, THREADS = Cfg::WARPS * 32;
  constexpr float kLift = kWeightLift<T>;
  constexpr unsigned kAll = 0xffffffffu;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* rings = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int worker = warp * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);   // few workers: one to an SM first
  uint8_t* ring = rings + warp * Cfg::RING;                                                     // stage: K tile, V tile
  uint64_t* full = reinterpret_cast<uint64_t*>(rings + Cfg::WARPS * Cfg::RING) + warp * ST;
  int* start = reinterpret_cast<int*>(rings + Cfg::WARPS * (Cfg::RING + ST * 8));
  int* row0 = start + b.n_seq + 2;
  int* len = row0 + b.n_seq + 1;
  const StreamDeal deal{start, row0, len};

  if (lane == 0) {
    for (int s = 0; s < ST; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  // the prefix kernel takes over SMs as this one leaves them; a join that came early would only wait
  // beside the scores (4 rows over 5120 keys: 14.7 us for 13.4)
  if (p.pre_tc) pdl_launch_dependents();
  {   // the page table and the queries on their way to L2 while the deal is found
    const int64_t i = static_cast<int64_t>(blockIdx.x) * THREADS + threadIdx.x, tables = static_cast<int64_t>(b.n_seq) * b.table_stride / 32;
    const int lines = a.Hq * D / 64;   // 128-byte lines of a row of q
    if (i < tables) prefetch_l2(b.page_table + i * 32);
    if (i < static_cast<int64_t>(b.n_rows) * lines) prefetch_l2(static_cast<const T*>(a.q) + i / lines * a.q_stride + i % lines * 64);
  }
  // ---- the deal: first tile of every sequence
  {
    __shared__ int64_t sums[Cfg::WARPS];
    const int per = (b.n_seq + THREADS - 1) / THREADS, s0 = threadIdx.x * per, s1 = min(b.n_seq, s0 + per);
    int64_t mine = 0;
    for (int s = s0; s < s1; ++s) {
      const SeqSpan q = seq_span(b, s);
      if (q.bad && blockIdx.x == 0) flag_status(status, QCF_DEV_BAD_INDEX);
      const int n = stream_tiles_of(q, a.G, c.Hkv);
      start[s] = n;
      row0[s] = q.row0;
      if (s == b.n_seq - 1) row0[s + 1] = b.row_start[s + 1];
      len[s] = q.len;
      mine += n;
    }
    int64_t run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(kAll, run, o);
      if (lane >= o) run += v;
    }
    if (lane == 31) sums[warp] = run;
    __syncthreads();
    const int pre = p.pre_stream ? p.stream_blocks * p.stream_tiles * c.Hkv : 0;
    int64_t all = pre, before = pre + run - mine;
    for (int w = 0; w < Cfg::WARPS; ++w) {
      all += sums[w];
      if (w < warp) before += sums[w];
    }
    // more tiles than the bounds allow come only of sequences that overlap: nothing is done for them
    const bool over = all > kMostTiles;
    if (over && blockIdx.x == 0 && threadIdx.x == 0) flag_status(status, QCF_DEV_BAD_INDEX);
    int at = over ? 0 : static_cast<int>(before);
    for (int s = s0; s < s1; ++s) {
      const int n = over ? 0 : start[s];
      start[s] = at;
      at += n;
    }
    if (threadIdx.x == THREADS - 1) {   // the last thread's end is the total
      start[b.n_seq] = at;
      start[b.n_seq + 1] = max((at + p.workers - 1) / p.workers, kMinShare);
    }
    __syncthreads();
    if (blockIdx.x == 0 && threadIdx.x == 0) *ws.share = start[b.n_seq + 1];
  }

  // ---- copies: a walk of its own, up to ST tiles ahead of the scores.  The lanes hold the page ids of
  // a window of 32 groups of 8 keys (8 tiles) of a unit, and those of the next window, asked for when
  // the window before began.
  StreamWalk ahead(b, p, deal, worker, c.Hkv);
  StreamSeg cs, ns;              // units of this window and the next
  int ci = 0, ni = 0, ids = 0, nids = 0, cn = 0;   // tile of the unit, page id of this lane's group; tiles issued
  unsigned out = 0, bad = 0;     // groups outside the cache: of the window, of the tiles issued (4 bits each, tile % 8)
  bool copies = ahead.next(cs, b, p, a, deal, c.Hkv), more = copies;
  StreamWalk walk = ahead;       // of the scores
  StreamSeg s = cs;
  bool live = copies;
  auto ask = [&](const StreamSeg& u, int i) {   // page ids of the window at tile i of u
    const int key = (u.t0 + i) * kStreamKeys + lane * 8;
    return key < u.len ? u.table[key >> c.page_shift] : c.n_pages;
  };
  auto next_window = [&]() {     // ns, ni: the window behind cs, ci
    ns = cs;
    ni = ci + 8;
    while (more && ni >= ns.use) {   // units without a tile to read are passed over
      more = ahead.next(ns, b, p, a, deal, c.Hkv);
      ni = 0;
    }
    if (more) nids = ask(ns, ni);
  };
  auto enter_window = [&]() {    // the ids of cs at tile ci: n_pages, which reads as zeros, behind the length or outside the cache
    const bool wrong = ids < 0 || ids > c.n_pages || (ids == c.n_pages && (cs.t0 + ci) * kStreamKeys + lane * 8 < cs.len);
    if (wrong) {
      flag_status(status, QCF_DEV_BAD_INDEX);
      ids = c.n_pages;
    }
    out = __ballot_sync(kAll, wrong);
  };
  const int ps = min(1 << c.page_shift, kStreamKeys), pages = kStreamKeys / ps;   // rows of a box, pages of a tile
  auto copy_next = [&]() {
    if (!copies) return;
    const int at = (cn & 7) * 4;
    bad = (bad & ~(15u << at)) | (out >> ((ci & 7) * 4) & 15u) << at;
    const int st = cn % ST, page = lane & 3, key0 = (cs.t0 + ci) * kStreamKeys;
    const int id = __shfl_sync(kAll, ids, (ci & 7) * 4 + page * (ps >> 3));
    if (lane == 0) mbar_arrive_expect_tx(&full[st], 2 * Cfg::TILE);
    __syncwarp();
    if (lane < 8 && page < pages) {   // lanes 0 .. 3: K, 4 .. 7: V
      uint8_t* dst = ring + (2 * st + (lane >> 2)) * Cfg::TILE + page * ps * Cfg::COLS * 2;
      const CUtensorMap* map = lane < 4 ? &tmK : &tmV;
#pragma unroll
      for (int h = 0; h < Cfg::BOXES; ++h)
        tma_load_4d(dst + h * Cfg::BOX, map, &full[st], h * Cfg::COLS, key0 & ((1 << c.page_shift) - 1), cs.g, id);
    }
    ++cn;
    ++ci;
    if ((ci & 7) == 0 || ci == cs.use) {
      copies = more;
      if (!copies) return;
      cs = ns;
      ci = ni;
      ids = nids;
      enter_window();
      next_window();
    }
  };
  const int mi = lane >> 3, mr = lane & 7, qc = (lane & 3) * 2, r_lo = lane >> 2;
  uint32_t qf[D / 16][4];
  auto load_q = [&](const StreamSeg& u) {
    const int end = min(u.rho0 + kStreamRows, u.nq * a.G), lo = u.rho0 + r_lo, hi = lo + 8;
    auto q_row = [&](int rho) {
      const int r = div_g(a, rho);
      return static_cast<const T*>(a.q) + static_cast<int64_t>(u.row0 + r) * a.q_stride +
             static_cast<int64_t>(u.g * a.G + rho - r * a.G) * D;
    };
    const T* ql = lo < end ? q_row(lo) : nullptr;
    const T* qh = hi < end ? q_row(hi) : nullptr;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      qf[ks][0] = ql ? *reinterpret_cast<const uint32_t*>(ql + ks * 16 + qc) : 0u;
      qf[ks][1] = qh ? *reinterpret_cast<const uint32_t*>(qh + ks * 16 + qc) : 0u;
      qf[ks][2] = ql ? *reinterpret_cast<const uint32_t*>(ql + ks * 16 + qc + 8) : 0u;
      qf[ks][3] = qh ? *reinterpret_cast<const uint32_t*>(qh + ks * 16 + qc + 8) : 0u;
    }
  };
  if (live) {
    while (more && ci >= cs.use) more = ahead.next(cs, b, p, a, deal, c.Hkv);   // the first unit with a tile to read
    copies = more;
    if (copies) ids = ask(cs, 0);
    load_q(s);
    if (copies) {
      enter_window();
      next_window();
    }
#pragma unroll
    for (int i = 0; i < ST; ++i) copy_next();
  }

  // what the join needs to know of each row, found while the first tiles come
  for (int64_t row = blockIdx.x + static_cast<int64_t>(gridDim.x) * threadIdx.x; row < b.n_rows; row += static_cast<int64_t>(gridDim.x) * THREADS) {
    int lo = -1, hi = b.n_seq;   // the last sequence that begins at or before the row
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (row0[mid] <= row) lo = mid; else hi = mid;
    }
    const bool real = lo >= 0 && row < row0[lo + 1] && start[lo + 1] > start[lo];
    ws.rows[row] = real ? make_int4(static_cast<int>(row) - row0[lo], start[lo], (len[lo] + kStreamKeys - 1) / kStreamKeys, 0) : make_int4(-1, 0, 0, 0);
  }

  // ---- scores
  int n = 0;
  bool ok = true;
  while (live) {
    const int end = min(s.rho0 + kStreamRows, s.nq * a.G), lo = s.rho0 + r_lo, hi = lo + 8;   // this thread's score rows
    // the last key a row sees: all of the prefix, or the own token of its position
    const int lim_lo = s.pre ? s.len : s.len - s.nq + div_g(a, lo), lim_hi = s.pre ? s.len : s.len - s.nq + div_g(a, hi);
    const int lim_min = s.pre ? s.len : s.len - s.nq + div_g(a, s.rho0);
    float m_lo = -INFINITY, m_hi = -INFINITY, l_lo = 0.f, l_hi = 0.f;
    float acc[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;

    for (int i = 0; i < s.use; ++i, ++n) {
      const int st = n % ST, kb = (s.t0 + i) * kStreamKeys;
      const unsigned gone = bad >> ((n & 7) * 4) & 15u;   // its groups of 8 keys outside the cache
      if (!__all_sync(kAll, mbar_wait(&full[st], (n / ST) & 1))) {
        ok = false;
        break;
      }
      uint8_t* k_tile = ring + 2 * st * Cfg::TILE;
      uint8_t* v_tile = k_tile + Cfg::TILE;
      const uint32_t ka = smem_u32(k_tile), va = smem_u32(v_tile);
      if (kb + kStreamKeys > s.len) {   // values behind the length: a free slot may hold NaN, and 0 x NaN is NaN
        for (int e = lane; e < kStreamKeys * (D / 8); e += 32) {
          const int key = e / (D / 8);
          if (kb + key >= s.len) *reinterpret_cast<uint4*>(v_tile + tile_at<D>(key, e % (D / 8) * 8)) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();   // before the stage's next copy
        __syncwarp();
      }
      float sc[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t b0, b1, b2, b3;
          ldsm_x4(ka + tile_at<D>(h * 16 + (mi >> 1) * 8 + mr, ks * 16 + (mi & 1) * 8), b0, b1, b2, b3);
          mma_16816<T>(sc[2 * h], qf[ks], b0, b1);
          mma_16816<T>(sc[2 * h + 1], qf[ks], b2, b3);
        }
      if (kb + kStreamKeys > s.len || kb + kStreamKeys - 1 > lim_min || gone) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = kb + j * 8 + qc + (e & 1);
            if (key >= s.len || key > (e < 2 ? lim_lo : lim_hi) || (gone >> j & 1)) sc[j][e] = -INFINITY;
          }
      }
      float top_lo = fmaxf(max3(sc[0][0], sc[0][1], sc[1][0]), max3(sc[1][1], sc[2][0], sc[2][1]));
      float top_hi = fmaxf(max3(sc[0][2], sc[0][3], sc[1][2]), max3(sc[1][3], sc[2][2], sc[2][3]));
      top_lo = max3(top_lo, sc[3][0], sc[3][1]) * a.scale_log2;
      top_hi = max3(top_hi, sc[3][2], sc[3][3]) * a.scale_log2;
      // rows of a quad share their maximum only when one of them asks for it
      if (__any_sync(kAll, top_lo > m_lo + (8.f + kLift) || top_hi > m_hi + (8.f + kLift))) {
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) {
          top_lo = fmaxf(top_lo, __shfl_xor_sync(kAll, top_lo, o));
          top_hi = fmaxf(top_hi, __shfl_xor_sync(kAll, top_hi, o));
        }
        const float n_lo = fmaxf(m_lo, top_lo - kLift), n_hi = fmaxf(m_hi, top_hi - kLift);
        const float f_lo = m_lo == -INFINITY ? 0.f : fast_exp2(m_lo - n_lo), f_hi = m_hi == -INFINITY ? 0.f : fast_exp2(m_hi - n_hi);
        m_lo = n_lo;
        m_hi = n_hi;
        l_lo *= f_lo;
        l_hi *= f_hi;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          acc[j][0] *= f_lo;
          acc[j][1] *= f_lo;
          acc[j][2] *= f_hi;
          acc[j][3] *= f_hi;
        }
      }
      const float b_lo = m_lo == -INFINITY ? 0.f : -m_lo, b_hi = m_hi == -INFINITY ? 0.f : -m_hi;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sc[j][0] = fast_exp2(fmaf(sc[j][0], a.scale_log2, b_lo));
        sc[j][1] = fast_exp2(fmaf(sc[j][1], a.scale_log2, b_lo));
        sc[j][2] = fast_exp2(fmaf(sc[j][2], a.scale_log2, b_hi));
        sc[j][3] = fast_exp2(fmaf(sc[j][3], a.scale_log2, b_hi));
        l_lo += sc[j][0] + sc[j][1];
        l_hi += sc[j][2] + sc[j][3];
      }
      // the weights meet the values in the cache's 16-bit type (the MMA's); their sum stays fp32
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t pa[4] = {pack2<T>(sc[2 * h][0], sc[2 * h][1]), pack2<T>(sc[2 * h][2], sc[2 * h][3]),
                                pack2<T>(sc[2 * h + 1][0], sc[2 * h + 1][1]), pack2<T>(sc[2 * h + 1][2], sc[2 * h + 1][3])};
#pragma unroll
        for (int dp = 0; dp < D / 16; ++dp) {
          uint32_t b0, b1, b2, b3;
          ldsm_x4_t(va + tile_at<D>(h * 16 + (mi & 1) * 8 + mr, dp * 16 + (mi >> 1) * 8), b0, b1, b2, b3);
          mma_16816<T>(acc[2 * dp], pa, b0, b1);
          mma_16816<T>(acc[2 * dp + 1], pa, b2, b3);
        }
      }
      __syncwarp();
      copy_next();   // into the stage that every lane has left
    }
    if (!ok) break;
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
      l_lo += __shfl_xor_sync(kAll, l_lo, o);
      l_hi += __shfl_xor_sync(kAll, l_hi, o);
    }

    // ---- the rows' sums leave, as a part or finished, while the next unit's queries come
    StreamSeg next;
    live = walk.next(next, b, p, a, deal, c.Hkv);
    if (live) load_q(next);
    const bool only = b.prefix_len == 0 && s.nt == s.tiles;
    float* part_o = s.part > 0 ? ws.spill_o + static_cast<int64_t>(worker) * kStreamRows * D : s.pre ? ws.pre_o : ws.own_o;
    float2* part_ml = s.part > 0 ? ws.spill_ml + static_cast<int64_t>(worker) * kStreamRows : s.pre ? ws.pre_ml : ws.own_ml;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int rho = half ? hi : lo;
      if (rho >= end) continue;
      const float m = half ? m_hi : m_lo, l = half ? l_hi : l_lo;
      const int r = div_g(a, rho);
      const int64_t place = static_cast<int64_t>(s.row0 + r) * a.Hq + s.g * a.G + rho - r * a.G;
      const int64_t slot = s.part > 0 ? static_cast<int64_t>(rho - s.rho0) : place;
      if (only) {
        const float inv = l > 0.f ? 1.f / l : 0.f;
        T* o = static_cast<T*>(a.o) + place * D;
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
          *reinterpret_cast<uint32_t*>(o + j * 8 + qc) = pack2<T>(acc[j][2 * half] * inv, acc[j][2 * half + 1] * inv);
        if (a.lse && qc == 0) a.lse[place] = (m + log2f(l)) * 0.69314718055994531f;
      } else {
        float* o = part_o + slot * D;
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
          *reinterpret_cast<float2*>(o + j * 8 + qc) = make_float2(acc[j][2 * half], acc[j][2 * half + 1]);
        if (qc == 0) part_ml[slot] = make_float2(m, l);
      }
    }
    s = next;
  }
  if (!ok) {
    flag_status(status, QCF_DEV_TIMEOUT);
    for (int e = n; e < cn; ++e) mbar_wait(&full[e % ST], (e / ST) & 1);   // no copy is in flight when the warp ends
  }
}

// ------------------------------------------------------------------ joining the parts
//
// A warp joins the parts of one head of a row: a lane has 16 bytes of each, and a batch of parts is
// loaded, sums and statistics together, before it is added with a running maximum.  `per` warps
// (1, 2, 4 or 8) share the parts where there may be many; their results meet in shared memory,
// always in the same order.  The parts of the tcgen05 prefix and the first of the own tokens have
// places that depend on the row alone, and are on their way while the row's deal is read.
// Bound by latencies: the end of the kernel before it, the row, a batch of parts, the next.  5 us
// for 2048 pairs of 15 parts and 4 for 128 of 80, against a join that returns at once; batches of 8,
// or more than 64 registers, took 2 to 4 us more of the former, two warps a pair 1.5.
constexpr int kCombineWarps = 8;
template <typename T, int D>
__global__ void __launch_bounds__(kCombineWarps * 32) batch_combine_kernel(const PagedView c, const BatchView b, const AttnArgs a,
                                                                           const SharedPlan p, const Workspace ws, int per) {
  constexpr int BATCH = 4;
  __shared__ float met[kCombineWarps][D + 2];   // a warp's sums, normaliser, maximum
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp % per;
  const unsigned unit = blockIdx.x * static_cast<unsigned>(kCombineWarps / per) + warp / per;
  const bool out = unit >= static_cast<unsigned>(b.n_rows) * a.Hq;   // behind the last pair: nothing to do, but for the barrier
  const int row = out ? 0 : static_cast<int>(unit / a.Hq), h = out ? 0 : static_cast<int>(unit - row * a.Hq);
  const int g = h / a.G, hh = h - g * a.G;
  const int64_t at = static_cast<int64_t>(row) * a.Hq + h;
  const bool has = lane * 4 < D;   // this lane's entries: 4 lane ..
  int known = 0;   // parts: the first of the own tokens, the prefix's, the others of the own tokens
  if (p.pre_even) {
    known = 1 + p.pre_parts;
  } else if (p.pre_tc) {   // the CTAs that share this row's unit
    const int u = g * p.pre_row_blocks + row / p.pre_rows;
    known = 2 + ((u + 1) * p.pre_tiles - 1) / p.pre_share - u * p.pre_tiles / p.pre_share;
  }
  pdl_wait();
  const int4 at_row = ws.rows[row];   // row of its sequence (-1: of none), the sequence's first tile, tiles of its length
  const int share = *ws.share;
  float M = -INFINITY, L = 0.f, sum[4] = {0.f, 0.f, 0.f, 0.f};
  // parts first, first + per, ... below end; place(i, o): its statistics, and its sums in o
  auto join = [&](int first, int end, auto place) {
    for (int i0 = first; i0 < end; i0 += per * BATCH) {
      float2 ml[BATCH];
      float4 v[BATCH];
#pragma unroll
      for (int j = 0; j < BATCH; ++j) {   // behind the end the last part again: loads without branches stay together
        const float* o;
        ml[j] = *place(min(i0 + per * j, end - 1), o);
        v[j] = *reinterpret_cast<const float4*>(o + (has ? lane * 4 : 0));
      }
#pragma unroll
      for (int j = 0; j < BATCH; ++j)
        if (i0 + per * j < end && ml[j].y != 0.f) {   // a part without keys for this row has no sums
          const float top = fmaxf(M, ml[j].x);
          const float f = fast_exp2(ml[j].x - top), e = M == -INFINITY ? 0.f : fast_exp2(M - top);
          M = top;
          L = fmaf(ml[j].y, f, L * e);
          sum[0] = fmaf(v[j].x, f, sum[0] * e);
          sum[1] = fmaf(v[j].y, f, sum[1] * e);
          sum[2] = fmaf(v[j].z, f, sum[2] * e);
          sum[3] = fmaf(v[j].w, f, sum[3] * e);
        }
    }
  };
  join(sub, known, [&](int i, const float*& o) {
    const int64_t r = i == 0 ? at : static_cast<int64_t>(i - 1) * b.n_rows * a.Hq + at;
    o = (i == 0 ? ws.own_o : ws.tc_o) + r * D;
    return (i == 0 ? ws.own_ml : ws.tc_ml) + r;
  });
  // by the deal: a streamed prefix, the other parts of the own tokens
  int n_pre = 0, n_own = 0, pre_cta = 0, pre_local = 0, own_cta = 0, rho = 0;
  if (at_row.x >= 0) {
    if (p.pre_stream) {
      const int r = row * a.G + hh, first = (r / kStreamRows * c.Hkv + g) * p.stream_tiles;
      pre_cta = first / share;
      pre_local = r % kStreamRows;
      n_pre = (first + p.stream_tiles - 1) / share - pre_cta + 1;
    }
    rho = at_row.x * a.G + hh;
    const int first = at_row.y + (rho / kStreamRows * c.Hkv + g) * at_row.z;
    own_cta = first / share;
    n_own = (first + at_row.z - 1) / share - own_cta + 1;
  }
  const int skip = known > 0 ? 1 : 0;   // the first of the own tokens' parts
  const bool done = out || known + n_pre + n_own <= 1 || at_row.x < 0;   // written already, or not a row of a sequence
  const int left = done ? 0 : n_pre + n_own - skip;
  join(sub, left, [&](int i, const float*& o) {
    const bool pre = i < n_pre;
    if (!pre) i += skip - n_pre;
    if (i == 0) {
      o = (pre ? ws.pre_o : ws.own_o) + at * D;
      return (pre ? ws.pre_ml : ws.own_ml) + at;
    }
    const int64_t r = static_cast<int64_t>((pre ? pre_cta : own_cta) + i) * kStreamRows + (pre ? pre_local : rho % kStreamRows);
    o = ws.spill_o + r * D;
    return ws.spill_ml + r;
  });
  if (per > 1) {
    if (has)
#pragma unroll
      for (int e = 0; e < 4; ++e) met[warp][lane * 4 + e] = sum[e];
    if (lane == 0) {
      met[warp][D] = L;
      met[warp][D + 1] = M;
    }
    __syncthreads();
    if (sub > 0) return;
    float top = -INFINITY;
    for (int w = 0; w < per; ++w) top = fmaxf(top, met[warp + w][D + 1]);
    M = top;
    L = sum[0] = sum[1] = sum[2] = sum[3] = 0.f;
    for (int w = 0; w < per; ++w) {
      const float mw = met[warp + w][D + 1], f = mw == -INFINITY ? 0.f : fast_exp2(mw - top);
      L = fmaf(met[warp + w][D], f, L);
      if (has)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] = fmaf(met[warp + w][lane * 4 + e], f, sum[e]);
    }
  }
  if (done || !has) return;
  const float inv = L > 0.f ? 1.f / L : 0.f;
  *reinterpret_cast<uint2*>(static_cast<T*>(a.o) + at * D + lane * 4) = make_uint2(pack2<T>(sum[0] * inv, sum[1] * inv), pack2<T>(sum[2] * inv, sum[3] * inv));
  if (a.lse && lane == 0) a.lse[at] = (M + log2f(L)) * 0.69314718055994531f;
}

// ------------------------------------------------------------------ host

static SharedPlan plan_shared(const PagedView& c, const BatchView& b, int Hq) {
  SharedPlan p = {};
  const int G = Hq / c.Hkv, sms = num_sms();
  p.ctas = sms;
  p.workers = sms * (c.D == 128 ? StreamCfg<128>::WARPS : c.D == 64 ? StreamCfg<64>::WARPS : StreamCfg<16>::WARPS);
  // The prefix goes to tcgen05 where more than one 16-row block of score rows shares it and its tiles
  // would be more than three to each warp of the stream; below that a kernel of its own costs more
  // than it saves.  32 query heads over 8 KV heads, head dim 128, in us (stream / tcgen05): 8 rows
  // and 1000 keys (0.6 tiles a warp) 14.3 / 19.3, 24 and 1000 (1.7) 19.0 / 20.8, 8 and 5120 (2.8)
  // 19.8 / 21.7, 24 and 3000 keys (4.9) 30.3 / 23.4, 64 and 3000 (13) 44.3 / 36.6.
  const int64_t blocks = (static_cast<int64_t>(b.n_rows) * G + kStreamRows - 1) / kStreamRows;
  const int64_t tiles = (static_cast<int64_t>(b.prefix_len) + kStreamKeys - 1) / kStreamKeys;
  if (c.D >= 64 && blocks > 1 && blocks * tiles * c.Hkv > 3 * static_cast<int64_t>(p.workers)) {
    p.pre_tc = true;
    p.pre_rows = 2 * (128 / G);
    p.pre_row_blocks = (b.n_rows + p.pre_rows - 1) / p.pre_rows;
    p.pre_tiles = (b.prefix_len + 127) / 128;
    const int64_t units = static_cast<int64_t>(p.pre_row_blocks) * c.Hkv, total = units * p.pre_tiles;
    p.pre_share = static_cast<int>(std::max<int64_t>((total + sms - 1) / sms, std::min(2, p.pre_tiles)));
    // Each unit in equal parts where that takes no CTA more than a tile longer (a second unit costs a
    // CTA about three): the KV heads then read the same rows at the same time, which share DRAM pages
    // (the call with 32 rows, 64 heads and 131072 keys 117.0 us, dealt out 120.4; with 64 rows, 32
    // heads and 5120 keys 36.7 and 40.3).
    const int each = units <= sms ? (p.pre_tiles + static_cast<int>(sms / units) - 1) / static_cast<int>(sms / units) : INT32_MAX;
    if (each <= p.pre_share + 1) {
      p.pre_even = true;
      p.pre_parts = (p.pre_tiles + std::max(each, p.pre_share) - 1) / std::max(each, p.pre_share);
      p.pre_ctas = static_cast<int>(units * p.pre_parts);
    } else {
      p.pre_ctas = static_cast<int>((total + p.pre_share - 1) / p.pre_share);
      p.pre_parts = (p.pre_tiles + p.pre_share - 2) / p.pre_share + 1;   // CTAs that one unit can meet
    }
  } else if (b.prefix_len > 0) {
    p.pre_stream = true;
    p.stream_blocks = static_cast<int>(blocks);
    p.stream_tiles = static_cast<int>(tiles);
  }
  return p;
}

// Tiles of the stream at most: every sequence as long as its bound, and as wide as its bound or as all rows allow.
static int64_t most_tiles(const SharedPlan& p, const BatchView& b, int G, int Hkv) {
  const int64_t rows = std::min(b.max_q, b.n_rows), blocks = b.n_seq * ((rows * G + kStreamRows - 1) / kStreamRows);
  const int64_t together = (static_cast<int64_t>(b.n_rows) * G + static_cast<int64_t>(b.n_seq) * (kStreamRows - 1)) / kStreamRows;
  return (static_cast<int64_t>(p.stream_blocks) * p.stream_tiles +
          std::min(blocks, together) * ((b.max_len + kStreamKeys - 1) / kStreamKeys)) *
         Hkv;
}

size_t workspace_layout(const SharedPlan& p, const BatchView& b, int Hq, int D, void* base, Workspace* w) {
  uint8_t* at = static_cast<uint8_t*>(base);
  size_t used = 0;
  auto take = [&](size_t bytes) {
    uint8_t* r = at + used;
    used += align_up(bytes, 256);
    return r;
  };
  const size_t rows = static_cast<size_t>(b.n_rows) * Hq, o = rows * D * sizeof(float), ml = rows * sizeof(float2);
  w->rows = reinterpret_cast<int4*>(take(static_cast<size_t>(b.n_rows) * sizeof(int4)));
  w->share = reinterpret_cast<int*>(take(sizeof(int)));
  w->tc_o = reinterpret_cast<float*>(take(p.pre_parts * o));
  w->tc_ml = reinterpret_cast<float2*>(take(p.pre_parts * ml));
  w->own_o = reinterpret_cast<float*>(take(o));
  w->own_ml = reinterpret_cast<float2*>(take(ml));
  w->pre_o = reinterpret_cast<float*>(take(p.pre_stream ? o : 0));
  w->pre_ml = reinterpret_cast<float2*>(take(p.pre_stream ? ml : 0));
  w->spill_o = reinterpret_cast<float*>(take(static_cast<size_t>(p.workers) * kStreamRows * D * sizeof(float)));
  w->spill_ml = reinterpret_cast<float2*>(take(static_cast<size_t>(p.workers) * kStreamRows * sizeof(float2)));
  return used;
}

template <typename T, int D>
static cudaError_t stream_launch(const CUtensorMap& tk, const CUtensorMap& tv, const PagedView& c, const BatchView& b,
                                 const AttnArgs& a, const SharedPlan& p, const Workspace& w, cudaStream_t st) {
  static PerDevice<cudaError_t> smem_attr;
  const cudaError_t attr = smem_attr.get(current_device(), [] {
    return cudaFuncSetAttribute(stream_attn_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(stream_smem<D>(kMaxBatchSeqs)));
  });
  if (attr != cudaSuccess) return attr;
  LaunchScope ls(KC_OWN_ATTN, st);
  // Not launch_pdl: that this kernel starts behind all earlier work is what lets it, and the prefix kernel
  // launched beside it, read queries and pages and write the scratch without a wait of their own.
  const dim3 grid(p.ctas), block(StreamCfg<D>::WARPS * 32);
  stream_attn_kernel<T, D><<<grid, block, stream_smem<D>(b.n_seq), st>>>(tk, tv, c, b, a, p, w, device_status_ptr());
  return cudaGetLastError();
}

template <typename T, int D>
static qcf_status shared_prefix_attn_launch(const qcf_paged_kv* cache, const PagedView& c, const BatchView& b, const AttnArgs& a,
                                            const SharedPlan& p, const Workspace& w, cudaStream_t st) {
  CUtensorMap tk, tv;
  const int rows = std::min(1 << c.page_shift, kStreamKeys);
  const CUtensorMapSwizzle sw = D >= 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE;
  if (!encode_pages(&tk, cache->k, c, rows, StreamCfg<D>::COLS, sw) || !encode_pages(&tv, cache->v, c, rows, StreamCfg<D>::COLS, sw))
    return set_error(QCF_ERR_CUDA, "qcf_shared_prefix_attn: tensor map encoding failed");
  cudaError_t e = stream_launch<T, D>(tk, tv, c, b, a, p, w, st);
  if (e != cudaSuccess) return cuda_error(e, "qcf_shared_prefix_attn: launch");
  if (p.pre_tc) {
    const qcf_status s = prefix_tc_launch(cache, c, b, a, p, w, st);
    if (s != QCF_OK) return s;
  }
  LaunchScope ls(KC_BATCH_COMBINE, st);
  // parts of a row, about (lengths are known on the device): a warp for every few of them
  const int64_t share = std::max<int64_t>(kMinShare, most_tiles(p, b, a.G, c.Hkv) / p.workers);
  const int64_t many = p.pre_parts + (p.stream_tiles + (b.max_len + kStreamKeys - 1) / kStreamKeys) / share + 1;
  const int per = many <= 16 ? 1 : many <= 32 ? 2 : many <= 64 ? 4 : 8;
  const int64_t pairs = static_cast<int64_t>(b.n_rows) * a.Hq, at_once = kCombineWarps / per;
  e = launch_pdl(batch_combine_kernel<T, D>, dim3(static_cast<unsigned>((pairs + at_once - 1) / at_once)), dim3(kCombineWarps * 32), 0,
                 st, c, b, a, p, w, per);
  return e == cudaSuccess ? QCF_OK : cuda_error(e, "qcf_shared_prefix_attn: combine launch");
}

template <typename T>
static qcf_status shared_prefix_attn_type(const qcf_paged_kv* cache, const PagedView& c, const BatchView& b, const AttnArgs& a,
                                          const SharedPlan& p, const Workspace& w, cudaStream_t st) {
  switch (c.D) {
    case 16: return shared_prefix_attn_launch<T, 16>(cache, c, b, a, p, w, st);
    case 64: return shared_prefix_attn_launch<T, 64>(cache, c, b, a, p, w, st);
    default: return shared_prefix_attn_launch<T, 128>(cache, c, b, a, p, w, st);
  }
}

static qcf_status check_attn(const char* who, const qcf_paged_kv* cache, const qcf_paged_batch* batch, int Hq, PagedView* c,
                             BatchView* b) {
  const qcf_status s = check_paged(who, cache, batch, c, b);
  if (s != QCF_OK) return s;
  if (b->n_seq > kMaxBatchSeqs) return set_error(QCF_ERR_SHAPE, "%s: n_seq=%d (at most %d)", who, b->n_seq, kMaxBatchSeqs);
  if (Hq <= 0 || Hq % c->Hkv || Hq / c->Hkv > 16) return set_error(QCF_ERR_SHAPE, "%s: Hq=%d Hkv=%d", who, Hq, c->Hkv);
  if (static_cast<int64_t>(b->n_rows) * Hq > INT32_MAX / 128)
    return set_error(QCF_ERR_SHAPE, "%s: %d rows of %d heads are too many for one call", who, b->n_rows, Hq);
  const SharedPlan p = plan_shared(*c, *b, Hq);
  if (most_tiles(p, *b, Hq / c->Hkv, c->Hkv) > kMostTiles || static_cast<int64_t>(p.pre_row_blocks) * c->Hkv * p.pre_tiles > kMostTiles)
    return set_error(QCF_ERR_SHAPE, "%s: the bounds allow more work than one call takes", who);
  return QCF_OK;
}

}  // namespace qcf

using namespace qcf;

extern "C" {

size_t qcf_shared_prefix_attn_workspace_size(const qcf_paged_kv* cache, const qcf_paged_batch* batch, int Hq) {
  PagedView c;
  BatchView b;
  if (check_attn("qcf_shared_prefix_attn_workspace_size", cache, batch, Hq, &c, &b) != QCF_OK) return 0;
  if (b.n_seq == 0 || b.n_rows == 0) return 0;
  Workspace w;
  return workspace_layout(plan_shared(c, b, Hq), b, Hq, c.D, nullptr, &w);
}

qcf_status qcf_shared_prefix_attn(const qcf_paged_kv* cache, const qcf_paged_batch* batch, const void* q, int64_t q_stride,
                                  int Hq, float scale, void* o, float* lse, void* ws, size_t ws_bytes, void* stream) {
  const char* who = "qcf_shared_prefix_attn";
  PagedView c;
  BatchView b;
  const qcf_status s = check_attn(who, cache, batch, Hq, &c, &b);
  if (s != QCF_OK) return s;
  if (!q || !o) return set_error(QCF_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (!(scale > 0.f) || !std::isfinite(scale * 1.4426950408889634f)) return set_error(QCF_ERR_INVALID_ARG, "%s: scale=%g", who, scale);
  if (q_stride < static_cast<int64_t>(Hq) * c.D)
    return set_error(QCF_ERR_SHAPE, "%s: q_stride %lld for %d x %d entries", who, (long long)q_stride, Hq, c.D);
  if (take_fault(4) || !aligned16(q) || !aligned16(o) || q_stride % 8 || (reinterpret_cast<uintptr_t>(ws) & 255u))
    return set_error(QCF_ERR_ALIGN, "%s: pointers and strides must be multiples of 16 bytes, ws of 256", who);
  // warps write finished rows of o while others still load the queries of other rows
  if (o == q && q_stride != static_cast<int64_t>(Hq) * c.D)
    return set_error(QCF_ERR_SHAPE, "%s: o is q, whose rows lie %lld entries apart instead of %d x %d", who, (long long)q_stride, Hq, c.D);
  if (take_fault(1)) return set_error(QCF_ERR_INVALID_ARG, "%s: injected invalid index table", who);
  if (take_fault(2)) return set_error(QCF_ERR_WORKSPACE, "%s: injected short workspace", who);
  if (b.n_seq == 0 || b.n_rows == 0) return QCF_OK;
  const SharedPlan p = plan_shared(c, b, Hq);
  Workspace w;
  const size_t need = workspace_layout(p, b, Hq, c.D, ws, &w);
  if (!ws || ws_bytes < need) return set_error(QCF_ERR_WORKSPACE, "%s: workspace %zu < %zu", who, ws_bytes, need);
  const AttnArgs a{q, q_stride, o, lse, Hq, Hq / c.Hkv,
                   static_cast<uint32_t>(((1ull << 32) + Hq / c.Hkv - 1) / (Hq / c.Hkv)), scale * 1.4426950408889634f};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return cache->dtype == QCF_BF16 ? shared_prefix_attn_type<__nv_bfloat16>(cache, c, b, a, p, w, st)
                                  : shared_prefix_attn_type<__half>(cache, c, b, a, p, w, st);
}

}  // extern "C"
