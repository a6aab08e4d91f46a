// Attention of many new tokens of a sequence at a time: whole prompts packed one behind the other,
// and chunks of prompts over a paged cache that holds them already.
//
// For a row at position p, o = sum_j w_j V_j / sum_j w_j with w_j = 2^(x_j - m), x_j = scale log2(e) q.K_j over
// the keys j <= p (and j > p - window), m a running maximum: one pass over the keys, the sums rescaled
// when m grows.
//
// Two CTAs of a cluster (a pair) work on one unit: up to four row tiles of 128 score rows (new rows x
// the G query heads of one KV head) of one sequence, against its key tiles of 128.  A product spans the pair
// (cta_group::2, 256 rows): row tile x = a, b of both CTAs at once, each holding half of every K
// tile (64 keys) and of every V tile (half of the columns).  That halves what a CTA loads, keeps and
// feeds to a product: with K and V whole in one CTA, S = Q K^T reads its operands at the full rate of
// shared memory (128 bytes a cycle for 64 cycles of products), which the arriving tiles then slow down.
//
// Twelve warps a CTA:
//   warp 0      walks the pair's share of the work and passes units on through a small ring; K producer by
//               tiled TMA (pages: one box per page and 64 columns), and Q
//   warp 2      V producer; rows behind a sequence's end are zeroed, since 0 x NaN is NaN
//   warps 1, 3  in the first CTA, one lane each issues the products of row tile x for both: P_x V, then
//               S_x = Q_x K^T of the next key tile, the two taking turns
//   warps 4-7   softmax of a, warps 8-11 of b: thread = score row of this CTA; the weights back to tensor
//               memory over the scores they came from, the output rescaled only when a row's maximum
//               grows by more than 2^8; the unit's output at its end
// A unit with rows in a alone (single tokens, short questions) takes its key tiles by turns: a has the
// even ones and b the odd ones of the same rows, and the output joins the two.
// Tensor memory columns: S_a 0, S_b 128 (the weights take the first 64 of each), O_a 256, O_b 256 + DP.
//
// Bound: a causal prompt of 17984 tokens, 64 heads over 8: 3.08 to 3.22 ms, 1.64 to 1.72 PFLOP/s (cuBLAS:
// 1.89 in bursts, 1.72 kept up under the power limit, where this kernel runs too).  A pair of row tiles takes
// 2550 to 2750 cycles a key tile, 2048 of them products.  One row tile's own chain is as long: S 512, its
// arrival 150, the softmax's two halves 1100 and 450, the arrival at the issuer 220, the last products 256.  Two row
// tiles are what fits tensor memory at head dim 128.  At 64, with half the products to the same softmax, that
// chain bounds: 2300 cycles by these figures, and the period is 2260 (16384 tokens, 32 heads over 8: 1071 us, 1.03
// PFLOP/s), while the tensor pipe, the powers and the issue slots are in use 40, 40 and 43 % of the time (8192 tokens).
// A unit costs another 5000 cycles (queries, the first scores, a masked tile, the output), which bounds many
// short prompts: ten of 512 tokens 37.4 us, floor 15.7.  Small calls: the launch 2.5 us, the deal 2.5, loads and one
// tile 4, code that is fetched as it runs the first time: four questions of up to 64 tokens 13.0 us.
#include <algorithm>
#include <cmath>

#include "paged_attn.cuh"

namespace qcf {

constexpr int kMaxChunkSeqs = 8000;   // the deal keeps 12 bytes of each where the rings will be
constexpr int kTileKeys = 128;
constexpr int kTileThreads = 384;
constexpr int kTileRows = 512;        // score rows of a unit
// The deal is by cost: so many for a unit, for a key tile of a unit with one row tile in use (1680 cycles), with both
// (2650), and for those of a group, whose own tiles come from pages met nowhere else.  (The mixed step below 273 us, dealt
// like other tiles 294, at 6 and 8 280; 1024 rows and 100 single tokens of up to 4000 own keys 277, 267, 319.)  A unit counts
// for no more than 2650 cycles here and takes 5000, so pairs with many short units get too much: by these cycles the longest
// pair has 33 us of work at 2048 tokens where the mean is 26, and 30 with a unit at 11.  Other values have not been measured.
constexpr int kUnitCost = 6, kTileCost1 = 4, kTileCost2 = 6, kGroupCost1 = 5, kGroupCost2 = 7;
// Tiles at least on each side of a cut through a unit: a cut costs the sums' way out and the join.  2 parts of 512
// rows: 8 us of the call.  When this was chosen, prompts of 1024 / 2048 / 4096 tokens, 64 rows over
// 5120 keys, in us: 3 tiles 26.8 / 52.0 / 123.1, 22.6; 4 24.7 / 51.3 / 122.4, 23.8; 6 21.9 / 51.9 / 118.0, 24.4; 8 21.9 / 52.2 / 117.2, 26.0.
constexpr int kMinCut = 3;
constexpr int kMinCost = 18;          // dealt to a pair at least
constexpr int kSegRing = 4;

// What the two entry points differ in: keys and values as rows of one tensor each, or in pages.
struct ChunkArgs {
  AttnArgs a;
  int D, window, per;   // per: tokens of a row tile
  int group;            // sequences of at most so many new rows share a prefix as a group; 0: none does
};
struct ChunkParts {     // units cut through: each pair may leave the end of one and the beginning of another
  int4* rec;            // [pairs]: parts of the unit that begins here and ends elsewhere (0: none), its first row, rows, KV head
  float2* ml;           // [pairs][2][kTileRows]
  float* o;             // [pairs][2][kTileRows][D]; rows of a unit: 128 to each of its row tiles
};

template <int DP>
struct TileCfg {
  static constexpr int BOXES = DP / 64;
  static constexpr int QBOX = 128 * 128, QTILE = BOXES * QBOX;          // a CTA's 128 score rows
  static constexpr int KBOX = 64 * 128, KTILE = BOXES * KBOX;           // its 64 keys
  static constexpr int VCOLS = DP / 2, VTILE = kTileKeys * VCOLS * 2;   // its columns of 128 values
  // 4 and one box of output: 3 and two take 1 % less where many rows share a tile, and 10 to 16 % more where few do
  // (8 questions of 33 to 64 rows over 16384 keys 123 us for 107, one row over 65536 70 for 59).
  static constexpr int STAGES = DP == 128 ? 4 : 8;
  static constexpr int OBOX = 128 * 128, OBOXES = DP == 128 ? 1 : 2, OTILE = OBOXES * OBOX;   // output: 128 bytes of 128 rows to a box
  static constexpr int FIXED = 3 * 1024;
  static constexpr int SMEM = 2 * QTILE + STAGES * (KTILE + VTILE) + 2 * OTILE + FIXED;
};
static_assert(TileCfg<128>::SMEM <= 232448 && TileCfg<64>::SMEM <= 232448, "227 KB of a CTA");

__device__ __forceinline__ SeqSpan chunk_span(const BatchView& b, int seq) {
  if (b.kv_len) return seq_span(b, seq);
  SeqSpan s;
  s.row0 = b.row_start[seq];
  const int end = b.row_start[seq + 1];
  s.bad = s.row0 < 0 || end < s.row0 || end > b.n_rows || end - s.row0 > b.max_q;
  s.nq = s.len = s.bad ? 0 : end - s.row0;
  return s;
}

// ------------------------------------------------------------------ pairs of CTAs

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The cluster address of what lies at this shared-memory address in CTA `rank`.
__device__ __forceinline__ uint32_t at_rank(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
// Arrivals at a barrier of either CTA.  What they announce lies in tensor memory or comes by TMA, which have
// ordering of their own: without a scope the arrival orders no other memory across the pair (a release for the
// cluster is a memory barrier of 500 cycles or more, and made every weight tile wait for it).
__device__ __forceinline__ void mbar_arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive_expect_tx_at(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void fence_cluster() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }
// Tiled loads to this CTA that count on a barrier of either (its cluster address).
__device__ __forceinline__ void tma_load_3d_pair(void* smem_dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
      ::"r"(smem_u32(smem_dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d_pair(void* smem_dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];"
      ::"r"(smem_u32(smem_dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* smem_src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];"
               ::"l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(smem_src)), "r"(x), "r"(y), "r"(z)
               : "memory");
}
// The shared memory of this thread's bulk stores has been read.
__device__ __forceinline__ void bulk_wait_read0() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
// Eight bits for each of the lowest four.
__device__ __forceinline__ uint32_t bytes_of(unsigned b) {
  return (b & 1u) * 0xffu | (b >> 1 & 1u) * 0xff00u | (b >> 2 & 1u) * 0xff0000u | (b >> 3 & 1u) * 0xff000000u;
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
}
// The lowest n bits, none below 0 and all from 32 on.
__device__ __forceinline__ uint32_t bits_below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)), "r"(ncols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// The products of umma_f16 and umma_f16_ts over 256 rows, 128 in each CTA; the descriptors hold in both.
// A whole warp runs the issuing code, so that descriptors stay in uniform registers, and `one` lane of it issues.
__device__ __forceinline__ void umma_f16_pair(bool one, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 e, %5, 0;\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(static_cast<uint32_t>(one))
      : "memory");
}
__device__ __forceinline__ void umma_f16_ts_pair(bool one, uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 e, %5, 0;\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(static_cast<uint32_t>(one))
      : "memory");
}
// umma_f16_ts_pair that leaves the rows with a set bit in `off` (128 of the first CTA, 128 of the second) as they are.
__device__ __forceinline__ void umma_f16_ts_pair_rows(bool one, uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, const uint32_t* off) {
  asm volatile(
      "{\n .reg .pred p, e;\n setp.eq.b32 p, 0, 0;\n setp.ne.b32 e, %4, 0;\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, {%5, %6, %7, %8, %9, %10, %11, %12}, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(static_cast<uint32_t>(one)), "r"(off[0]), "r"(off[1]), "r"(off[2]), "r"(off[3]), "r"(off[4]),
      "r"(off[5]), "r"(off[6]), "r"(off[7])
      : "memory");
}
// Arrives on this barrier in both CTAs once every product issued by this thread is complete.
__device__ __forceinline__ void umma_commit_pair(bool one, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred e;\n setp.ne.b32 e, %2, 0;\n"
      " @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}\n" ::"r"(smem_u32(bar)),
      "h"(static_cast<uint16_t>(3)), "r"(static_cast<uint32_t>(one))
      : "memory");
}
// 32 lanes x 16 consecutive 32-bit columns from registers into tensor memory; tmem_wait_st() before others may read them.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])),
      "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])),
      "r"(__float_as_uint(v[8])), "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
      "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])), "r"(__float_as_uint(v[15]))
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// sdesc_mnmajor_sw128 for rows of 32 entries: 64-byte swizzle, atoms of 8 rows in 512 bytes.
__device__ __forceinline__ uint64_t sdesc_mnmajor_sw64(uint32_t smem_addr) {
  return static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4) | static_cast<uint64_t>(1u) << 16 | static_cast<uint64_t>(512u >> 4) << 32 |
         static_cast<uint64_t>(1u) << 46 | static_cast<uint64_t>(4u) << 61;
}

// ------------------------------------------------------------------ the deal
//
// The units of all sequences, row block by row block and KV head by KV head, lie one behind the other
// on a line, each as long as its cost.  Pair i takes what lies between i and i + 1 shares of it; a border
// that falls into a unit cuts it between two key tiles, or is moved to its nearer end where fewer than
// kMinCut tiles would lie on one side.

// A run of sequences with a few new rows each (single tokens) within 32 aligned ones goes as a group: its
// rows lie side by side in the batch and make one unit, which reads the shared prefix once for all of them and
// then each one's own tiles, which the rows of the others do not see: their weights are 0, and their sums
// are left out of the product, for 0 x NaN is NaN and one sequence's values must not spoil another.  (44
// single tokens of 32 heads over a prefix of 5120 tokens, in five runs beside four chunks of 3172 together: 271 us for the
// call, 402 with a unit to each at an earlier step.)  It stands in the place of its
// first sequence; its length is kept as -1 - (32 own tiles + (sequences - 1)).
struct Span {
  int row0, nq, len;   // nq 0: no rows, or those of a group that began before
};
__device__ __forceinline__ int group_size(int len) { return ((-1 - len) & 31) + 1; }
__device__ __forceinline__ int group_tiles(int len) { return (-1 - len) >> 5; }
__device__ __forceinline__ int warp_scan(int v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (static_cast<int>(threadIdx.x & 31) >= o) v += u;
  }
  return v;
}
// Of sequence base + lane, base a multiple of 32; all lanes of a warp together.
template <bool GROUPS>
__device__ __forceinline__ Span span_at(const BatchView& b, const ChunkArgs& p, int base, bool* bad) {
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31, seq = base + lane;
  SeqSpan q = {0, 0, 0, false};
  if (seq < b.n_seq) q = chunk_span(b, seq);
  *bad = q.bad;
  Span s{q.row0, q.nq, q.len};
  if (!GROUPS) return s;
  const bool small = seq < b.n_seq && !q.bad && q.nq <= p.group;
  const unsigned in = __ballot_sync(kAll, small), rows = __ballot_sync(kAll, small && q.nq > 0);
  const int tiles = small && q.nq > 0 ? (q.len + kTileKeys - 1) / kTileKeys : 0;
  const int nq_sum = warp_scan(small ? q.nq : 0), tile_sum = warp_scan(tiles);
  const unsigned gap_below = ~in & ((1u << lane) - 1u), gap_above = ~in >> lane;
  const int first = 32 - __clz(gap_below), end = gap_above ? lane + __ffs(gap_above) - 1 : 32;   // the run of this lane
  const int nq_run = __shfl_sync(kAll, nq_sum, max(end - 1, 0)) - nq_sum + q.nq;
  const int tile_run = __shfl_sync(kAll, tile_sum, max(end - 1, 0)) - tile_sum + tiles;
  const unsigned run = small ? (0xffffffffu >> (32 - (end - first))) << first : 0u;
  if (__popc(rows & run) < 2) return s;
  if (lane == first) return Span{q.row0, nq_run, -1 - (tile_run * 32 + end - first - 1)};
  return Span{q.row0, 0, q.len};
}

struct RowBlock {
  int i0, ntok;            // tokens of the sequence
  int t0, end, end_a;      // its key tiles; the end of row tile a's
  int cost;                // of a key tile
  __device__ int tiles() const { return end - t0; }
};
__device__ __forceinline__ int tile_of(int prefix, int pos) {
  return pos < prefix ? pos / kTileKeys : (prefix + kTileKeys - 1) / kTileKeys + (pos - prefix) / kTileKeys;
}
__device__ __forceinline__ bool two_tiles(const RowBlock& k, int per) { return k.ntok > 2 * per; }
template <bool GROUPS>
__device__ __forceinline__ RowBlock row_block(const BatchView& b, const ChunkArgs& p, int nq, int len, int i) {
  RowBlock k;
  k.i0 = i * 4 * p.per;
  k.ntok = min(4 * p.per, nq - k.i0);
  if (GROUPS && len < 0) {
    k.t0 = 0;
    k.end = k.end_a = (b.prefix_len + kTileKeys - 1) / kTileKeys + group_tiles(len);
    k.cost = two_tiles(k, p.per) ? kGroupCost2 : kGroupCost1;
    return k;
  }
  const int pos = b.prefix_len + len - nq + k.i0;   // of its first token
  k.t0 = p.window ? tile_of(b.prefix_len, max(0, pos - p.window + 1)) : 0;
  k.end = tile_of(b.prefix_len, pos + k.ntok - 1) + 1;
  k.end_a = tile_of(b.prefix_len, pos + min(k.ntok, 2 * p.per) - 1) + 1;
  k.cost = two_tiles(k, p.per) ? kTileCost2 : kTileCost1;
  return k;
}
__device__ __forceinline__ int unit_cost(const RowBlock& k) { return kUnitCost + k.cost * k.tiles(); }
// The tile of a unit before which a border at cost x behind its beginning cuts it.
__device__ __forceinline__ int cut_at(const RowBlock& k, int x) {
  const int n = k.tiles(), t = min(max(x - kUnitCost, 0) / k.cost, n);
  return t < kMinCut ? 0 : n - t < kMinCut ? n : t;
}

struct DealStart {
  int seq, block;       // seq -1: nothing for this pair
  int pos, share;       // cost before the row block
  int row0, nq, len;    // of the sequence or group
  int unused;
};

// One unit, or the part of one, of this pair.
struct Segment {
  int seq, row0, ntok, g;      // its first row in the batch, its tokens
  int pos, len;                // own position of its first token; own tokens of the sequence (or a group's, see Span)
  int t0, nt, nt_a, nt_b;      // first key tile, tiles, those of row tiles a and b
  int split;                   // 1: no rows in b, so it takes the odd tiles of a's rows, a the even ones
  int slot;                    // -1: the whole unit, else where its sums go
  int end;                     // 1: there are no more
};

// What comes from memory is alike in all lanes of a warp, which the compiler cannot see: from one lane it knows, and keeps
// addresses, descriptors and loop bounds once for the warp instead of once for each lane (17984 tokens 3.30 -> 3.16 ms).
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }
__device__ __forceinline__ void make_uniform(Segment& s) {
  s.seq = uniform(s.seq);
  s.row0 = uniform(s.row0);
  s.ntok = uniform(s.ntok);
  s.g = uniform(s.g);
  s.pos = uniform(s.pos);
  s.len = uniform(s.len);
  s.t0 = uniform(s.t0);
  s.nt = uniform(s.nt);
  s.nt_a = uniform(s.nt_a);
  s.nt_b = uniform(s.nt_b);
  s.split = uniform(s.split);
  s.slot = uniform(s.slot);
}

// The deal is found by the softmax warps, while others set up barriers and tensor memory.
constexpr int kDealThreads = 256;
__device__ __forceinline__ void deal_sync() { bar_sync(7, kDealThreads); }
// Sum over the threads before this one, and over all; met: 8 ints of its own for each use.
__device__ __forceinline__ int deal_scan(int tid, int v, int* met, int* total) {
  const int warp = tid >> 5, lane = tid & 31;
  int run = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += u;
  }
  if (lane == 31) met[warp] = run;
  deal_sync();
  int before = run - v;
  *total = 0;
#pragma unroll
  for (int w = 0; w < kDealThreads / 32; ++w) {
    const int u = met[w];
    *total += u;
    if (w < warp) before += u;
  }
  return before;
}

// Finds where this pair's share begins; blk: scratch for 3 n_seq + 1 ints.
template <bool GROUPS>
__device__ void find_share(int tid, const BatchView& b, const ChunkArgs& p, int Hkv, int pair, int pairs, int* blk, int* met, DealStart* start,
                           unsigned int* status) {
  const int R = 4 * p.per, most = b.n_rows / R + b.n_seq;   // row blocks at most
  const int per_s = (b.n_seq + kDealThreads - 1) / kDealThreads;
  const int s0 = min(b.n_seq, tid * per_s), s1 = min(b.n_seq, s0 + per_s);
  int* nqs = blk + b.n_seq + 1;
  int* lens = nqs + b.n_seq;
  int mine = 0, all, total;
  for (int s = tid; s - (tid & 31) < b.n_seq; s += kDealThreads) {
    bool bad;
    const Span q = span_at<GROUPS>(b, p, s - (tid & 31), &bad);
    if (bad && blockIdx.x == 0) flag_status(status, QCF_DEV_BAD_INDEX);
    if (s < b.n_seq) {
      blk[s] = (q.nq + R - 1) / R;
      nqs[s] = q.nq;
      lens[s] = q.len;
    }
  }
  deal_sync();
  for (int s = s0; s < s1; ++s) mine = min(mine + blk[s], most + 1);
  int at = deal_scan(tid, mine, met, &all);   // no overflow: 256 (most + 1) < 2^31
  // more row blocks than the rows allow come only of sequences that overlap: nothing is done for them
  const bool over = all > most;
  if (over && blockIdx.x == 0 && tid == 0) flag_status(status, QCF_DEV_BAD_INDEX);
  const int blocks = over ? 0 : all;
  for (int s = s0; s < s1; ++s) {
    const int n = blk[s];
    blk[s] = at;
    at += n;
  }
  if (tid == 0) {
    blk[b.n_seq] = blocks;
    start->seq = -1;
  }
  deal_sync();
  const int per_b = (blocks + kDealThreads - 1) / kDealThreads;
  const int b0 = min(blocks, tid * per_b), b1 = min(blocks, b0 + per_b);
  int first = 0;
  if (b0 < b1) {   // the last sequence that begins at or before block b0
    int hi = b.n_seq;
    while (hi - first > 1) {
      const int mid = (first + hi) >> 1;
      if (blk[mid] <= b0) first = mid; else hi = mid;
    }
  }
  // visit(seq, block of it, cost of the block's units)
  auto walk = [&](auto visit) {
    int seq = first;
    for (int i = b0; i < b1; ++i) {
      while (i >= blk[seq + 1]) ++seq;
      if (visit(seq, i - blk[seq], Hkv * unit_cost(row_block<GROUPS>(b, p, nqs[seq], lens[seq], i - blk[seq])))) return;
    }
  };
  int cost = 0;
  walk([&](int, int, int c) {
    cost += c;
    return false;
  });
  int pos = deal_scan(tid, cost, met + 8, &total);
  const int share = max((total + pairs - 1) / pairs, kMinCost);
  const int64_t want = static_cast<int64_t>(pair) * share;
  if (pos <= want && want < pos + cost)
    walk([&](int seq, int i, int c) {
      if (want >= pos + c) {
        pos += c;
        return false;
      }
      *start = DealStart{seq, i, pos, share, b.row_start[seq], nqs[seq], lens[seq], 0};
      return true;
    });
}

// Walks a pair's share, all lanes of a warp alike; they keep the spans of 32 sequences.
template <bool GROUPS>
struct TileWalk {
  const BatchView& b;
  const ChunkArgs& p;
  const int Hkv, pair;
  int pos, begin, stop, share;
  int seq, block, g, base;      // base: of the 32 sequences kept
  int my_row0, my_nq, my_len;   // this lane's
  int row0, nq, len;            // of seq
  RowBlock k;
  bool live;
  int4 rec;

  __device__ void keep(int from) {
    base = from;
    bool bad;
    const Span s = span_at<GROUPS>(b, p, from, &bad);
    my_row0 = s.row0;
    my_nq = s.nq;
    my_len = s.len;
  }
  __device__ void enter() {
    row0 = __shfl_sync(0xffffffffu, my_row0, seq - base);
    nq = __shfl_sync(0xffffffffu, my_nq, seq - base);
    len = __shfl_sync(0xffffffffu, my_len, seq - base);
  }
  __device__ TileWalk(const BatchView& b_, const ChunkArgs& p_, const DealStart& at, int Hkv_, int pair_) : b(b_), p(p_), Hkv(Hkv_), pair(pair_) {
    rec = make_int4(0, 0, 0, 0);
    live = at.seq >= 0;
    if (!live) return;
    pos = at.pos;
    share = at.share;
    begin = pair * share;
    stop = begin + share;
    seq = at.seq;
    block = at.block;
    keep(seq & ~31);
    row0 = at.row0;
    nq = at.nq;
    len = at.len;
    k = row_block<GROUPS>(b, p, nq, len, block);
    g = (begin - pos) / unit_cost(k);
    pos += g * unit_cost(k);
  }
  // The next sequence with rows.
  __device__ void next_seq() {
    while (true) {
      const unsigned rows = __ballot_sync(0xffffffffu, my_nq > 0), later = seq + 1 - base < 32 ? rows & (0xffffffffu << (seq + 1 - base)) : 0u;
      if (later) {
        seq = base + __ffs(later) - 1;
        enter();
        return;
      }
      if (base + 32 >= b.n_seq) {
        live = false;
        return;
      }
      keep(base + 32);
      seq = base - 1;
    }
  }
  __device__ bool next(Segment& s) {
    while (live) {
      const int n = k.tiles();
      const int cost = unit_cost(k);
      const int from = pos < begin ? cut_at(k, begin - pos) : 0, to = pos + cost > stop ? cut_at(k, stop - pos) : n;
      const bool some = from < to;
      if (some) {
        const bool two = two_tiles(k, p.per);
        s.seq = seq;
        s.row0 = row0 + k.i0;
        s.ntok = k.ntok;
        s.g = g;
        s.pos = GROUPS && len < 0 ? 0 : len - nq + k.i0;
        s.len = len;
        s.t0 = k.t0 + from;
        s.nt = to - from;
        s.split = !two;
        s.nt_a = two ? max(0, min(k.end_a - k.t0, to) - from) : (s.nt + 1) / 2;
        s.nt_b = two ? s.nt : s.nt / 2;
        s.slot = from == 0 && to == n ? -1 : from > 0 ? 0 : 1;
        s.end = 0;
        if (s.slot == 1) {   // how many borders cut this unit: those of the pairs behind this one
          int parts = 1;
          for (int at = stop; at < pos + cost; at += share) {
            const int t = cut_at(k, at - pos);
            parts += t > 0 && t < n;
          }
          rec = make_int4(parts, s.row0, s.ntok, g);
        }
      }
      pos += cost;
      if (pos >= stop) {
        live = false;
      } else if (++g == Hkv) {
        g = 0;
        if (++block * 4 * p.per >= nq) {
          block = 0;
          next_seq();
        }
        if (live) k = row_block<GROUPS>(b, p, nq, len, block);
      }
      if (some) return true;
    }
    return false;
  }
};

// ------------------------------------------------------------------ the kernel

template <typename T>
constexpr uint32_t idesc_pair(int N, bool b_mn_major) {
  return std::is_same<T, __half>::value ? idesc_bf16_f32(256, N, b_mn_major) & ~((1u << 7) | (1u << 10)) : idesc_bf16_f32(256, N, b_mn_major);
}

// GROUPS: a kernel of its own, for what groups need in the issuing warps costs other calls 1 to 4 %.
template <typename T, int DP, bool PAGED, bool GROUPS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kTileThreads, 1)
    tile_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmO, const __grid_constant__ CUtensorMap tmP, const PagedView c, const BatchView b,
                     const ChunkArgs p, const ChunkParts parts, unsigned int* status) {
  using Cfg = TileCfg<DP>;
  constexpr int ST = Cfg::STAGES;
  constexpr unsigned kAll = 0xffffffffu;
  const AttnArgs& a = p.a;
  extern __shared__ __align__(1024) uint8_t qbuf[];
  uint8_t* kbuf = qbuf + 2 * Cfg::QTILE;
  uint8_t* vbuf = kbuf + ST * Cfg::KTILE;
  uint8_t* obuf = vbuf + ST * Cfg::VTILE;
  float2* donated = reinterpret_cast<float2*>(obuf + 2 * Cfg::OTILE);   // [128]: maximum and sum of a's rows for b
  Segment* segs = reinterpret_cast<Segment*>(donated + 128);
  DealStart* start = reinterpret_cast<DealStart*>(segs + kSegRing);
  int* met = reinterpret_cast<int*>(start + 1);
  // in the first CTA, for both: what its issuers wait for
  uint64_t* k_full = reinterpret_cast<uint64_t*>(met + 16);
  uint64_t* v_full = k_full + ST;
  uint64_t* q_full = v_full + ST;
  uint64_t* p_ready = q_full + 1;    // [a, b][first, last 64 keys]
  // in each CTA
  uint64_t* k_empty = p_ready + 4;
  uint64_t* v_empty = k_empty + ST;
  uint64_t* q_empty = v_empty + ST;
  uint64_t* s_full = q_empty + 1;    // [a, b]
  uint64_t* o_done = s_full + 2;     // [a, b]
  uint64_t* mma_end = o_done + 2;    // [a, b]
  uint64_t* v_tail = mma_end + 2;
  uint64_t* seg_full = v_tail + 1;
  uint64_t* seg_empty = seg_full + kSegRing;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(seg_empty + kSegRing);
  static_assert(sizeof(Segment) * kSegRing % 8 == 0 && sizeof(DealStart) % 8 == 0, "barriers");
  static_assert(128 * 8 + sizeof(Segment) * kSegRing + sizeof(DealStart) + 64 + (4 * ST + 24 + 2 * kSegRing) * 8 <= Cfg::FIXED, "fixed part");

  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank()), pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmO);
    for (int s = 0; s < ST; ++s) {
      mbar_init(&k_full[s], 2);
      mbar_init(&v_full[s], 2);
      mbar_init(&k_empty[s], 2);
      mbar_init(&v_empty[s], 2);
    }
    mbar_init(q_full, 2);
    mbar_init(q_empty, 2);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&p_ready[2 * x], 9);       // the softmax warps of both CTAs and the turn
      mbar_init(&p_ready[2 * x + 1], 8);
      mbar_init(&s_full[x], 1);
      mbar_init(&o_done[x], 1);
      mbar_init(&mma_end[x], 1);
    }
    mbar_init(v_tail, 1);
    for (int s = 0; s < kSegRing; ++s) {
      mbar_init(&seg_full[s], 1);
      mbar_init(&seg_empty[s], rank == 0 ? 11 : 9);   // V producer, softmax warps, issuers
    }
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, 512);
  pdl_wait();
  if (warp >= 4) {
    find_share<GROUPS>(threadIdx.x - 128, b, p, c.Hkv, pair, pairs, reinterpret_cast<int*>(kbuf), met, start, status);
    fence_proxy_async_smem();   // the deal used the rings
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int np = (b.prefix_len + kTileKeys - 1) / kTileKeys;   // tiles of the prefix
  // A role's next segment; false when a wait ran out.
  int seg_n = 0;
  auto next_segment = [&](Segment& s) {
    const int at = seg_n % kSegRing;
    // longer than the walk's own waits take to run out: it still passes an end on, so that all warps see the same segments
    bool there = false;
    for (int i = 0; i < 5 && !there; ++i) there = mbar_wait(&seg_full[at], (seg_n / kSegRing) & 1);
    if (!there) return false;
    s = segs[at];
    ++seg_n;
    return true;
  };
  auto release_segment = [&] { mbar_arrive(&seg_empty[(seg_n - 1) % kSegRing]); };

  // The sequences of a grouped unit, one to a lane: own tokens, first own tile, first token in the unit, new rows.
  int sub_len = 0, sub_tile = 0, sub_tok = 0, sub_nq = 0;
  auto open_group = [&](const Segment& s) {
    if (!GROUPS || s.len >= 0) return;
    int tiles = 0;
    sub_tok = 0x7fffffff;
    if (lane < group_size(s.len)) {
      const SeqSpan q = seq_span(b, s.seq + lane);
      sub_len = q.len;
      sub_tok = q.row0 - s.row0;
      sub_nq = q.nq;
      tiles = q.nq > 0 ? (q.len + kTileKeys - 1) / kTileKeys : 0;
    }
    sub_tile = warp_scan(tiles) - tiles;
  };
  struct KeyTile {
    int seq;        // whose own tokens (-1: the prefix)
    int key0, len;  // its first key; keys there are
  };
  auto key_tile = [&](const Segment& s, int t) {
    if (t < np) return KeyTile{-1, t * kTileKeys, b.prefix_len};
    if (!GROUPS || s.len >= 0) return KeyTile{s.seq, (t - np) * kTileKeys, s.len};
    const int sub = max(__popc(__ballot_sync(kAll, lane < group_size(s.len) && sub_tile <= t - np)) - 1, 0);
    return KeyTile{s.seq + sub, (t - np - __shfl_sync(kAll, sub_tile, sub)) * kTileKeys, __shfl_sync(kAll, sub_len, sub)};
  };
  auto pages_of_tile = [&](const KeyTile& k) { return k.seq < 0 ? b.prefix_pages : b.page_table + static_cast<int64_t>(k.seq) * b.table_stride; };

  if (warp < 4) {
    // 88 x 128 + 208 x 256 threads: the 168 x 384 registers of the launch
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 0 || warp == 2) {
      // ---- the walk, K and Q; V
      const bool is_k = warp == 0;
      uint8_t* ring = is_k ? kbuf : vbuf;
      uint64_t* empty = is_k ? k_empty : v_empty;
      const uint32_t full = at_rank(is_k ? k_full : v_full, 0), q_full0 = at_rank(q_full, 0);
      constexpr int TILE_K = Cfg::KTILE, TILE_V = Cfg::VTILE;
      const int keys = is_k ? 64 : kTileKeys, key0 = is_k ? rank * 64 : 0;   // of a tile, in this CTA
      const int rows = PAGED ? min(1 << c.page_shift, keys) : keys, boxes = PAGED ? keys / rows : 1;
      DealStart at0 = *start;
      if (!is_k) at0.seq = -1;
      TileWalk<GROUPS> walk(b, p, at0, c.Hkv, pair);
      Segment s;
      int n = 0, tails = 0, units = 0;
      bool ok = true;
      while (ok) {
        if (is_k) {
          const bool more = walk.next(s);
          s.end = !more;
          const int at = seg_n % kSegRing;
          if (!__all_sync(kAll, mbar_wait(&seg_empty[at], ((seg_n / kSegRing) & 1) ^ 1u))) {
            ok = false;
            break;
          }
          if (lane == 0) {
            segs[at] = s;
            mbar_arrive(&seg_full[at]);
          }
          ++seg_n;
        } else {
          if (!__all_sync(kAll, next_segment(s))) {
            ok = false;
            break;
          }
          __syncwarp();
          if (lane == 0) release_segment();
        }
        if (s.end) break;
        make_uniform(s);
        open_group(s);
        // this lane's page of a tile: its id, n_pages (which reads as zeros) where there is none
        auto page_of = [&](const KeyTile& k) {
          const int key = k.key0 + key0 + lane * rows;
          if (lane >= boxes || key >= k.len) return c.n_pages;
          const int id = pages_of_tile(k)[key >> c.page_shift];
          if (id >= 0 && id < c.n_pages) return id;
          flag_status(status, QCF_DEV_BAD_INDEX);
          return c.n_pages;
        };
        KeyTile ahead = key_tile(s, s.t0);
        int next_id = PAGED ? page_of(ahead) : 0;
        for (int i = 0; i < s.nt; ++i, ++n) {
          const int st = n % ST, id = next_id;
          const KeyTile k = ahead;
          if (i + 1 < s.nt) {
            ahead = key_tile(s, s.t0 + i + 1);
            if (PAGED) next_id = page_of(ahead);
          }
          if (!__all_sync(kAll, mbar_wait(&empty[st], ((n / ST) & 1) ^ 1u))) {
            ok = false;
            break;
          }
          const int tk = k.key0, valid = k.len - tk;
          const int stale = valid < kTileKeys ? (PAGED ? min(kTileKeys, (valid + rows - 1) / rows * rows) : kTileKeys) : valid;
          const bool tail = !is_k && stale > valid;        // rows of the tile that lie behind the end
          const uint32_t bar = tail ? at_rank(v_tail, rank) : full + st * 8;
          uint8_t* dst = ring + st * (is_k ? TILE_K : TILE_V);
          if (lane == 0) mbar_arrive_expect_tx_at(bar, is_k ? TILE_K : TILE_V);
          __syncwarp();
          if (lane < boxes) {
            if (is_k) {
#pragma unroll
              for (int h = 0; h < Cfg::BOXES; ++h) {
                if constexpr (PAGED)
                  tma_load_4d_pair(dst + h * Cfg::KBOX + lane * rows * 128, &tmK, bar, h * 64, (tk + key0) & ((1 << c.page_shift) - 1), s.g, id);
                else
                  tma_load_3d_pair(dst + h * Cfg::KBOX, &tmK, bar, h * 64, s.g, s.row0 - s.pos + tk + key0);
              }
            } else {
              if constexpr (PAGED)
                tma_load_4d_pair(dst + lane * rows * Cfg::VCOLS * 2, &tmV, bar, rank * Cfg::VCOLS, tk & ((1 << c.page_shift) - 1), s.g, id);
              else
                tma_load_3d_pair(dst, &tmV, bar, rank * Cfg::VCOLS, s.g, s.row0 - s.pos + tk);
            }
          }
          if (is_k && i == 0) {   // the unit's Q: rows behind the sequence belong to others or are zeros, and go nowhere
            if (!__all_sync(kAll, mbar_wait(q_empty, (units & 1) ^ 1u))) {
              ok = false;
              break;
            }
            if (lane == 0) mbar_arrive_expect_tx_at(q_full0, 2 * Cfg::BOXES * p.per * a.G * 128);
            __syncwarp();
            if (lane < 2 * Cfg::BOXES)
              tma_load_3d_pair(qbuf + lane * Cfg::QBOX, &tmQ, q_full0, lane % Cfg::BOXES * 64, s.g * a.G,
                               s.row0 + (s.split ? rank : 2 * (lane / Cfg::BOXES) + rank) * p.per);
            ++units;
          }
          if (tail) {
            if (!__all_sync(kAll, mbar_wait(v_tail, tails++ & 1))) {
              ok = false;
              break;
            }
            constexpr int CH = Cfg::VCOLS / 8;   // 16-byte pieces of a row
            for (int e = lane; e < (stale - valid) * CH; e += 32)
              *reinterpret_cast<uint4*>(dst + valid * Cfg::VCOLS * 2 + e * 16) = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              fence_cluster();   // the zeros are written by ordinary stores, and the first CTA issues what reads them
              mbar_arrive_at(full + st * 8);
            }
          }
        }
      }
      if (!ok && lane == 0) flag_status(status, QCF_DEV_TIMEOUT);
      if (!ok && is_k) {
        const int at = seg_n % kSegRing;
        if (__all_sync(kAll, mbar_wait(&seg_empty[at], ((seg_n / kSegRing) & 1) ^ 1u)) && lane == 0) {
          segs[at].end = 1;
          mbar_arrive(&seg_full[at]);
        }
      }
      if (rank == 0) {   // no copy of this warp, or its like in the other CTA, is in flight when the CTAs end
        for (int e = max(0, n - ST); e < n; ++e)
          if (!mbar_wait(&(is_k ? k_full : v_full)[e % ST], (e / ST) & 1) && lane == 0) flag_status(status, QCF_DEV_TIMEOUT);
        if (is_k && units > 0 && !mbar_wait(q_full, (units - 1) & 1) && lane == 0) flag_status(status, QCF_DEV_TIMEOUT);
        if (is_k && lane == 0 && parts.rec) parts.rec[pair] = walk.rec;
      }
    } else if (rank == 0) {
      // ---- MMA issuer of row tile x of both CTAs
      const int x = warp >> 1;
      const bool one = lane == 0;
      constexpr uint32_t idesc_s = idesc_pair<T>(kTileKeys, false);
      constexpr uint32_t idesc_o = idesc_pair<T>(DP, true);
      constexpr int V_STEP = 16 * Cfg::VCOLS * 2;   // 16 keys of V
      int n = 0, k = 0;    // key tiles, segments so far
      uint32_t used = 0;   // weight tiles taken so far
      bool ok = true;
      Segment s;
      const uint64_t q_desc = sdesc_kmajor_sw128(smem_u32(qbuf + x * Cfg::QTILE));
      const uint64_t k_desc = sdesc_kmajor_sw128(smem_u32(kbuf));
      const uint64_t v_desc = DP == 128 ? sdesc_mnmajor_sw128(smem_u32(vbuf), 16) : sdesc_mnmajor_sw64(smem_u32(vbuf));
      const uint32_t q_empty1 = at_rank(q_empty, 1);
      // The turn: the barrier of a tile's first weights also counts one arrival of the other issuer,
      // made four products (256 cycles) before the end of its block, which covers what this warp
      // then takes to see it.
      auto pass = [&](bool due) {
        if (due && one) mbar_arrive(&p_ready[2 * (1 - x)]);
      };
      auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(kAll, mbar_wait(bar, parity)) != 0; };
      auto wait_k = [&](int tile) { return wait(&k_full[tile % ST], (tile / ST) & 1); };
      auto wait_v = [&](int tile) { return wait(&v_full[tile % ST], (tile / ST) & 1); };
      auto scores = [&](int tile, bool due, bool last) {   // S_x = Q_x K^T
        const uint64_t kd = k_desc + tile % ST * (Cfg::KTILE >> 4);
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk) {
          if (kk == DP / 16 - 4) pass(due);
          const uint64_t q_at = ((kk >> 2) * Cfg::QBOX + (kk & 3) * 32) >> 4, k_at = ((kk >> 2) * Cfg::KBOX + (kk & 3) * 32) >> 4;
          umma_f16_pair(one, tmem + x * 128, q_desc + q_at, kd + k_at, idesc_s, kk > 0 ? 1u : 0u);
        }
        umma_commit_pair(one, &s_full[x]);
        umma_commit_pair(one, &k_empty[tile % ST]);
        if (last) umma_commit_pair(one, q_empty);
      };
      while (true) {
        if (!(ok = __all_sync(kAll, next_segment(s)))) break;
        __syncwarp();
        if (one) release_segment();
        if (s.end) break;
        make_uniform(s);
        const int t0 = s.t0, nt = s.nt, nt_a = s.nt_a, nt_b = s.nt_b, mine = x ? nt_b : nt_a, split = s.split, step = 1 + split;
        open_group(s);
        if (!(ok = wait(q_full, k++ & 1))) break;
        // Every use of a stage is emptied by both issuers, also by the one whose row tile does not see the tile: that
        // one hands it on as soon as it is there.
        auto hand_k = [&](int tile) {
          if (!wait_k(tile)) return false;
          umma_commit_pair(one, &k_empty[tile % ST]);
          return true;
        };
        auto hand_v = [&](int tile) {
          if (!wait_v(tile)) return false;
          umma_commit_pair(one, &v_empty[tile % ST]);
          return true;
        };
        auto hand = [&](int tile) { return tile >= n + nt || (hand_k(tile) && hand_v(tile)); };
        const bool late = split && x;   // b's tiles of a split unit begin with the second
        int at = n + late;              // tile
        if (late && !(ok = hand_k(n))) break;
        if (mine > 0) {
          if (!(ok = wait_k(at))) break;
          tc_fence_after();
          scores(at, false, mine == 1);
        } else if (one) {
          mbar_arrive(q_empty);
          mbar_arrive_at(q_empty1);
        }
        if (late && !(ok = hand_v(n))) break;
        if (split && !(ok = hand(at + 1))) break;
        // of a group or not, told apart outside the loop: a choice in it costs other units 4 %
        auto tiles = [&](auto in_group) {
          constexpr bool IN_GROUP = decltype(in_group)::value;
          for (int i = 0; i < mine; ++i) {
            const bool more = i + 1 < mine;
            if (!(ok = wait_v(at))) break;
            const KeyTile kt = key_tile(s, t0 + at - n);
            if (kt.len - kt.key0 < kTileKeys) fence_cluster();   // zeros of the V producers
            const uint64_t vd = v_desc + at % ST * (Cfg::VTILE >> 4);
            const bool others = IN_GROUP && t0 + at - n >= np;   // others: rows that do not see these keys
            uint32_t off[8];
            if (others) {
              const int sub = kt.seq - s.seq, tok = __shfl_sync(kAll, sub_tok, sub), tok_end = tok + __shfl_sync(kAll, sub_nq, sub);
  #pragma unroll
              for (int w = 0; w < 8; ++w) {
                const int t0 = (split ? w >> 2 : 2 * x + (w >> 2)) * p.per, row0 = 32 * (w & 3);   // the row tile's first token, the word's first row
                const uint32_t on = bits_below((min(tok_end, t0 + p.per) - t0) * a.G - row0) & ~bits_below((tok - t0) * a.G - row0);
                off[w] = __reduce_or_sync(kAll, ~on);   // the same in all lanes: this leaves it in a uniform register, which the products take
              }
            }
            const uint32_t onto = IN_GROUP || i > 0 ? 1u : 0u;   // the softmax warps have cleared the sums of a group
            auto weigh = [&](int half) {   // O_x += P_x V over 64 keys
              tc_fence_after();
              if (others) {
  #pragma unroll
                for (int kk = half * (kTileKeys / 32); kk < (half + 1) * (kTileKeys / 32); ++kk)
                  umma_f16_ts_pair_rows(one, tmem + 256 + x * DP, tmem + x * 128 + kk * 8, vd + kk * (V_STEP >> 4), idesc_o, off);
                return;
              }
  #pragma unroll
              for (int kk = half * (kTileKeys / 32); kk < (half + 1) * (kTileKeys / 32); ++kk)
                umma_f16_ts_pair(one, tmem + 256 + x * DP, tmem + x * 128 + kk * 8, vd + kk * (V_STEP >> 4), idesc_o, kk > 0 ? 1u : onto);
            };
            // a begins, b follows while a has tiles left; who is alone gives itself the turn
            if ((x == 0 ? i == 0 : i >= nt_a) && one) mbar_arrive(&p_ready[2 * x]);
            const bool due = x == 0 ? i < nt_b : i + 1 < nt_a;
            if (!(ok = wait(&p_ready[2 * x], used & 1))) break;
            weigh(0);
            if (!(ok = wait(&p_ready[2 * x + 1], used & 1))) break;
            weigh(1);
            ++used;
            if (more) {
              if (!(ok = wait_k(at + step))) break;
              scores(at + step, due, i + 2 == mine);
            } else {
              pass(due);
              umma_commit_pair(one, &o_done[x]);
            }
            umma_commit_pair(one, &v_empty[at % ST]);   // after the scores: a commit costs more than a product
            if (split && more && !(ok = hand(at + 3))) break;
            at += step;
          }
        };
        if constexpr (GROUPS) {
          if (s.len < 0) tiles(std::true_type{}); else tiles(std::false_type{});
        } else {
          tiles(std::false_type{});
        }
        if (!ok) break;
        if (!split)
          for (; at < n + nt && ok; ++at) ok = hand(at);
        if (!ok) break;
        n += nt;
      }
      if (!ok && one) flag_status(status, QCF_DEV_TIMEOUT);
      umma_commit_pair(one, &mma_end[x]);   // nothing runs on tensor memory once it is freed
    }
  } else {
    // ---- softmax: thread = score row of tile x
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int x = (warp - 4) >> 2, quarter = warp & 3;
    const int rho = quarter * 32 + lane, pl = div_g(a, rho);
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_tm = tmem + lane_base + x * 128, o_tm = tmem + lane_base + 256 + x * DP;
    const uint32_t ready = at_rank(p_ready, 0) + 16 * x;
    uint8_t* obox = obuf + x * Cfg::OTILE;   // the tile's boxes of output
    uint32_t seen = 0, ends = 0;
    bool ok = true, stored = false;
    Segment s;
    while (true) {
      if (!__all_sync(kAll, next_segment(s))) {
        ok = false;
        break;
      }
      __syncwarp();
      if (lane == 0) release_segment();
      if (s.end) break;
      make_uniform(s);
      const int mine = x ? s.nt_b : s.nt_a, step = 1 + s.split, t_mine = s.t0 + (s.split & x);
      const int place = s.split ? rank : 2 * x + rank;   // of the row tile in the unit
      // this row's token, sequence and own position (a row of none: the last token's)
      const int tok = place * p.per + pl;
      int seq = s.seq, own = s.pos + min(tok, s.ntok - 1);
      open_group(s);
      if (GROUPS && s.len < 0) {
        int sub = 0;
        const int mine_tok = min(tok, s.ntok - 1);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
          if (__shfl_sync(kAll, sub_tok, sub + o) <= mine_tok) sub += o;
        seq = s.seq + sub;
        own = __shfl_sync(kAll, sub_len, sub) - __shfl_sync(kAll, sub_nq, sub) + mine_tok - __shfl_sync(kAll, sub_tok, sub);
        if (mine > 0) {   // own tiles leave other rows' sums as they are: all begin with 0
#pragma unroll 1
          for (int cc = 0; cc < DP / 16; ++cc) {
            const float zero[16] = {};
            tmem_st16(o_tm + cc * 16, zero);
          }
          tmem_wait_st();
          tc_fence_before();   // a warp that sees nothing of the first tile hands it on without another
        }
      }
      auto page_bad = [&](const KeyTile& k) {   // the page of this lane's 8 keys of a tile lies outside the cache
        const int key = k.key0 + lane * 8;
        if (lane >= kTileKeys / 8 || key >= k.len) return false;
        const int id = pages_of_tile(k)[key >> c.page_shift];
        return id < 0 || id >= c.n_pages;
      };
      float m = -INFINITY, l = 0.f;
      KeyTile ahead = key_tile(s, t_mine);
      bool bad = PAGED && mine > 0 && page_bad(ahead);
      for (int i = 0; i < mine; ++i) {
        const KeyTile k = ahead;
        const unsigned bad8 = PAGED ? __ballot_sync(kAll, bad) : 0u;
        if (i + 1 < mine) {
          ahead = key_tile(s, t_mine + (i + 1) * step);
          if constexpr (PAGED) bad = page_bad(ahead);
        }
        ok = ok && __all_sync(kAll, mbar_wait(&s_full[x], seen++ & 1));   // a warp whose wait ran out still meets the others
        tc_fence_after();
        // keys of the tile that this row sees: [low, high)
        const int high = k.seq < 0 ? k.len - k.key0 : k.seq == seq ? own + 1 - k.key0 : 0;
        if (GROUPS && k.seq >= 0 && s.len < 0 && !__any_sync(kAll, seq == k.seq)) {   // others' keys: the products leave the warp's rows out
          if (lane == 0) {
            mbar_arrive_at(ready);
            mbar_arrive_at(ready + 8);
          }
          continue;
        }
        float sv[kTileKeys];
        tmem_ld128(s_tm, sv);
        const int low = p.window ? (k.seq < 0 ? b.prefix_len : 0) + own + 1 - p.window - k.key0 : 0;
        if (__any_sync(kAll, high < kTileKeys || low > 0 || bad8)) {
          // one bit to each key: 800 cycles; comparisons of every key with both ends took 1500, skipping keys by eights more
#pragma unroll
          for (int w = 0; w < kTileKeys / 32; ++w) {
            uint32_t see = bits_below(high - 32 * w) & ~bits_below(low - 32 * w);
            if constexpr (PAGED) see &= ~bytes_of(bad8 >> (4 * w));
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!(see >> j & 1u)) sv[32 * w + j] = -INFINITY;
          }
        }
        float mx[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
        for (int j = 4; j < kTileKeys - 4; j += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], sv[j + e], sv[j + 4 + e]);
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], sv[kTileKeys - 4 + e]);
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
        const bool grow = top > m + (8.0f + kWeightLift<T>);
        if (__any_sync(kAll, grow)) {
          const float m_new = grow ? top - kWeightLift<T> : m;
          if (i > 0) {   // the full S of this tile says that every earlier product has been added to O
            const float f = m == -INFINITY ? 0.f : fast_exp2(m - m_new);
#pragma unroll 1
            for (int cc = 0; cc < DP / 16; ++cc) {
              float ov[16];
              tmem_ld16(o_tm + cc * 16, ov);
#pragma unroll
              for (int e = 0; e < 16; ++e) ov[e] *= f;
              tmem_st16(o_tm + cc * 16, ov);
            }
            tmem_wait_st();
            l *= f;
          }
          m = m_new;
        }
        // The weights leave in two halves, so that P V of the first 64 keys runs under the powers of the others.
        const float base = m == -INFINITY ? 0.f : -m;
        const Pair scale2 = make_pair2(a.scale_log2, a.scale_log2), base2 = make_pair2(base, base);
        Pair sum[2];
        sum[0] = sum[1] = make_pair2(0.f, 0.f);
#pragma unroll
        for (int part = 0; part < 4; ++part) {
          float pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int j = part * 32 + 2 * e;
            float p0, p1;
            split(fma2(make_pair2(sv[j], sv[j + 1]), scale2, base2), p0, p1);
            p0 = fast_exp2(p0);
            p1 = fast_exp2(p1);
            sum[e & 1] = add2(sum[e & 1], make_pair2(p0, p1));
            pk[e] = __uint_as_float(pack2<T>(p0, p1));
          }
          tmem_st16(s_tm + part * 16, pk);
          if (part & 1) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_at(ready + 8 * (part >> 1));
          }
        }
        float l0, l1;
        split(add2(sum[0], sum[1]), l0, l1);
        l += l0 + l1;
      }

      // ---- the unit's output
      const int rows = min(max(s.ntok - place * p.per, 0), p.per) * a.G;   // score rows of this CTA's tile
      const bool cut = s.slot >= 0, real = rho < rows, few = rows <= 32;
      const bool tiled = !few && (cut || rows == p.per * a.G);             // stored by whole tiles, all four warps together
      const int64_t first = static_cast<int64_t>(s.row0 + place * p.per) * a.Hq + s.g * a.G;            // head of score row 0
      const int64_t part = ((static_cast<int64_t>(pair) * 2 + max(s.slot, 0)) * 4 + place) * 128;       // cut: row 0 of the tile's sums
      uint8_t* out = obox + quarter * 32 * 128;   // this warp's rows of the first box
      auto boxes_free = [&] {   // tiled stores have read the boxes
        if (rho == 0) bulk_wait_read0();
        bar_sync(1 + x, 128);
      };
      if (stored) boxes_free();
      stored = false;
      if (mine > 0) {
        ok = ok && __all_sync(kAll, mbar_wait(&o_done[x], ends++ & 1));
        tc_fence_after();
      }
      float mine_f = 1.f, other_f = 0.f;
      if (s.split) {   // b takes a's sums, too
        if (x == 0) {
          donated[rho] = make_float2(m, l);
          tc_fence_before();
          bar_sync(3 + quarter, 64);
          bar_sync(3 + quarter, 64);   // they have been read
          tc_fence_after();            // a group's sums are cleared next
          continue;
        }
        bar_sync(3 + quarter, 64);
        tc_fence_after();
        const float2 ml = donated[rho];
        const float top = fmaxf(m, ml.x);
        mine_f = m == -INFINITY ? 0.f : fast_exp2(m - top);
        other_f = ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - top);
        l = l * (m == -INFINITY ? 1.f : mine_f) + ml.y * (ml.x == -INFINITY ? 1.f : other_f);   // without keys: 0, or NaN
        m = top;
      }
      if (real) {
        if (cut)
          parts.ml[part + rho] = make_float2(m, l);
        else if (a.lse)
          a.lse[first + static_cast<int64_t>(pl) * a.Hq + rho - pl * a.G] = (m + log2f(l)) * 0.69314718055994531f;
      }
      if (!cut) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        mine_f *= inv;
        other_f *= inv;
      }
      stored = tiled;
      // None of this warp's.  Tiled stores are made by all four warps together, whose barriers have to be as many, so there it
      // goes on like the others: what it writes lies behind the box of a whole tile (at 43 to 48 and 65 to 96 score rows a
      // token), or in sums of a cut one that the join does not read.
      if (!tiled && rows <= quarter * 32) {
        if (s.split) bar_sync(3 + quarter, 64);
        continue;
      }
#pragma unroll 1
      for (int c0 = 0; c0 < DP; c0 += 64) {
        float ov[64];
        tmem_ld64(o_tm + c0, ov);
        // nothing of b without a tile of its own, or where this part of a unit has none for a
#pragma unroll
        for (int e = 0; e < 64; ++e) ov[e] = mine > 0 ? ov[e] * mine_f : 0.f;
        if (s.split) {
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            float oa[16];
            tmem_ld16(tmem + lane_base + 256 + c0 + h * 16, oa);   // a has a tile at least
#pragma unroll
            for (int e = 0; e < 16; ++e) ov[h * 16 + e] = fmaf(oa[e], other_f, ov[h * 16 + e]);
          }
        }
        if (c0 + 64 >= DP) {
          tc_fence_before();
          if (s.split) bar_sync(3 + quarter, 64);
        }
        if (few) {   // rows go straight out
          if (real && cut) {
            float* o = parts.o + (part + rho) * p.D + c0;
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (c0 + e * 4 < p.D) *reinterpret_cast<float4*>(o + e * 4) = make_float4(ov[4 * e], ov[4 * e + 1], ov[4 * e + 2], ov[4 * e + 3]);
          } else if (real) {
            T* o = static_cast<T*>(a.o) + (first + static_cast<int64_t>(pl) * a.Hq + rho - pl * a.G) * p.D + c0;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (c0 + e * 8 < p.D) *reinterpret_cast<uint4*>(o + e * 8) = pack8<T>(ov + 8 * e);
          }
        } else if (cut && Cfg::OBOXES == 1) {   // 32 columns of 32 bits at a time
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (c0 + h > 0) boxes_free();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float* f = ov + 32 * h + 4 * e;
              *reinterpret_cast<float4*>(out + sw128_off(lane, e)) = make_float4(f[0], f[1], f[2], f[3]);
            }
            fence_proxy_async_smem();
            bar_sync(1 + x, 128);
            if (rho == 0 && c0 + 32 * h < p.D) {
              tma_store_2d(&tmP, obox, c0 + 32 * h, static_cast<int>(part));
              bulk_commit_group();
            }
          }
        } else if (cut) {   // or two boxes of them
#pragma unroll
          for (int e = 0; e < 16; ++e)
            *reinterpret_cast<float4*>(out + (e >> 3) * Cfg::OBOX + sw128_off(lane, e & 7)) = make_float4(ov[4 * e], ov[4 * e + 1], ov[4 * e + 2], ov[4 * e + 3]);
          fence_proxy_async_smem();
          bar_sync(1 + x, 128);
          if (rho == 0) {
            tma_store_2d(&tmP, obox, c0, static_cast<int>(part));
            if (c0 + 32 < p.D) tma_store_2d(&tmP, obox + Cfg::OBOX, c0 + 32, static_cast<int>(part));
            bulk_commit_group();
          }
        } else {
          if (Cfg::OBOXES == 1 && tiled && c0 > 0) boxes_free();
#pragma unroll
          for (int e = 0; e < 8; ++e) *reinterpret_cast<uint4*>(out + sw128_off(lane, e)) = pack8<T>(ov + 8 * e);
          if constexpr (Cfg::OBOXES == 1) {
            if (tiled) {   // every row of the tile: stores that run on while the next unit does
              fence_proxy_async_smem();
              bar_sync(1 + x, 128);
              if (rho == 0) {
                tma_store_3d(&tmO, obox, c0, s.g * a.G, s.row0 + place * p.per);
                bulk_commit_group();
              }
            } else {       // rows behind the sequence's end belong to others
              __syncwarp();
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int r = e * 4 + (lane >> 3), row = quarter * 32 + r, col = c0 + (lane & 7) * 8, tl = div_g(a, row);
                if (row < rows && col < p.D)
                  *reinterpret_cast<uint4*>(static_cast<T*>(a.o) + (first + static_cast<int64_t>(tl) * a.Hq + row - tl * a.G) * p.D + col) =
                      *reinterpret_cast<const uint4*>(out + sw128_off(r, lane & 7));
              }
              __syncwarp();
            }
          }
        }
      }
      if (Cfg::OBOXES == 1 || few || cut) continue;   // head dim 64: all columns in one box, after the loop (in it, as above, the call takes 7 % more)
      if (tiled) {   // every row of the tile: stores that run on while the next unit does
        fence_proxy_async_smem();
        bar_sync(1 + x, 128);
        if (rho == 0) {
#pragma unroll
          for (int h = 0; h < Cfg::BOXES; ++h)
            tma_store_3d(&tmO, obox + h * Cfg::OBOX, h * 64, s.g * a.G, s.row0 + place * p.per);
          bulk_commit_group();
        }
      } else {       // rows behind the sequence's end belong to others
        __syncwarp();
#pragma unroll 1
        for (int h = 0; h < Cfg::BOXES; ++h)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int r = e * 4 + (lane >> 3), row = quarter * 32 + r, col = h * 64 + (lane & 7) * 8, tl = div_g(a, row);
            if (row < rows && col < p.D)
              *reinterpret_cast<uint4*>(static_cast<T*>(a.o) + (first + static_cast<int64_t>(tl) * a.Hq + row - tl * a.G) * p.D + col) =
                  *reinterpret_cast<const uint4*>(out + h * Cfg::OBOX + sw128_off(r, lane & 7));
          }
        __syncwarp();
      }
    }
    if (rho == 0) bulk_wait_group0();   // the stores are done before this kernel counts as complete
    if (!ok && lane == 0) flag_status(status, QCF_DEV_TIMEOUT);
  }
  pdl_launch_dependents();   // the join comes up as pairs end
  tc_fence_before();
  __syncthreads();
  // in both CTAs: the commits that arrive here have all done so when the last has
  if (threadIdx.x < 2 && !mbar_wait(&mma_end[threadIdx.x], 0)) flag_status(status, QCF_DEV_TIMEOUT);
  __syncwarp();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ------------------------------------------------------------------ joining the parts
//
// A warp joins the parts of one score row of a unit that was cut: the one that its first pair left, and
// those of the pairs behind it.  The rows of all cut units, few or many, are dealt out over the warps.
// (A CTA to every 16 rows that a pair might have left: the call with 64 rows over 5120 keys 26.7 us for 22.2.)
constexpr int kJoinThreads = 256, kMaxPairs = kJoinThreads;
template <typename T>
__global__ void __launch_bounds__(kJoinThreads) tile_join_kernel(const ChunkArgs p, const ChunkParts parts, int pairs) {
  constexpr int WARPS = kJoinThreads / 32, BATCH = 8;
  __shared__ int4 rec_s[kMaxPairs];
  __shared__ int first_s[kMaxPairs + 1];   // rows of cut units before each pair's
  __shared__ int sums[WARPS];
  const AttnArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  {
    const int4 rec = static_cast<int>(threadIdx.x) < pairs ? parts.rec[threadIdx.x] : make_int4(0, 0, 0, 0);
    const int mine = rec.x > 1 ? rec.z * a.G : 0;
    const int run = warp_scan(mine);
    if (lane == 31) sums[warp] = run;
    rec_s[threadIdx.x] = rec;
    __syncthreads();
    int before = run - mine;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) before += w < warp ? sums[w] : 0;
    first_s[threadIdx.x] = before;
    if (threadIdx.x == kJoinThreads - 1) first_s[kMaxPairs] = before + mine;
    __syncthreads();
  }
  const int total = first_s[kMaxPairs];
  const bool has = lane * 4 < p.D;
  for (int row = blockIdx.x * WARPS + warp; row < total; row += gridDim.x * WARPS) {
    int pair = 0;   // the last one whose rows begin at or before this one: rows there are only of pairs that cut a unit
#pragma unroll
    for (int o = kMaxPairs / 2; o > 0; o >>= 1)
      if (first_s[pair + o] <= row) pair += o;
    const int4 rec = rec_s[pair];
    const int r = row - first_s[pair], tok = div_g(a, r), tile = tok / p.per, in_unit = tile * 128 + r - tile * p.per * a.G;
    float M = -INFINITY, L = 0.f, sum[4] = {0.f, 0.f, 0.f, 0.f};
    for (int i0 = 0; i0 < rec.x; i0 += BATCH) {
      float2 ml[BATCH];
      float4 v[BATCH];
#pragma unroll
      for (int j = 0; j < BATCH; ++j) {   // behind the end the last part again: loads without branches stay together
        const int i = min(i0 + j, rec.x - 1);
        const int64_t at = (static_cast<int64_t>(pair + i) * 2 + (i == 0 ? 1 : 0)) * kTileRows + in_unit;
        ml[j] = parts.ml[at];
        v[j] = *reinterpret_cast<const float4*>(parts.o + at * p.D + (has ? lane * 4 : 0));
      }
#pragma unroll
      for (int j = 0; j < BATCH; ++j)
        if (i0 + j < rec.x && ml[j].y != 0.f) {   // a part without keys for this row has no sums
          const float top = fmaxf(M, ml[j].x);
          const float f = ml[j].x == -INFINITY ? 1.f : fast_exp2(ml[j].x - top), e = M == -INFINITY ? 0.f : fast_exp2(M - top);
          M = top;
          L = fmaf(ml[j].y, f, L * e);
          sum[0] = fmaf(v[j].x, f, sum[0] * e);
          sum[1] = fmaf(v[j].y, f, sum[1] * e);
          sum[2] = fmaf(v[j].z, f, sum[2] * e);
          sum[3] = fmaf(v[j].w, f, sum[3] * e);
        }
    }
    const int64_t at = static_cast<int64_t>(rec.y + tok) * a.Hq + rec.w * a.G + r - tok * a.G;
    const float inv = L == 0.f ? 0.f : 1.f / L;
    if (has)
      *reinterpret_cast<uint2*>(static_cast<T*>(a.o) + at * p.D + lane * 4) = make_uint2(pack2<T>(sum[0] * inv, sum[1] * inv), pack2<T>(sum[2] * inv, sum[3] * inv));
    if (a.lse && lane == 0) a.lse[at] = (M + log2f(L)) * 0.69314718055994531f;
  }
}

// ------------------------------------------------------------------ host

// Key tiles of a unit at most.
static int64_t most_tiles(const BatchView& b) {
  return (static_cast<int64_t>(b.prefix_len) + kTileKeys - 1) / kTileKeys + (static_cast<int64_t>(b.max_len) + kTileKeys - 1) / kTileKeys;
}
// New rows of a sequence that may go in a group (0: none does): where a prefix of four tiles or more is read once for the
// group, and 32 of them fill no more than a unit.  max_len: the length of a Span holds its own tiles.
static int group_rows(const BatchView& b, int window, int per) {
  return window == 0 && b.n_seq > 1 && b.prefix_len >= 4 * kTileKeys && b.max_len <= 1 << 27 ? 4 * per / 32 : 0;
}
// Whether the bounds allow a unit long enough to be cut.
static bool may_cut(const BatchView& b, int window, int group) {
  int64_t tiles = most_tiles(b);
  if (window) tiles = std::min(tiles, (static_cast<int64_t>(window) + kTileRows + kTileKeys - 1) / kTileKeys + 2);
  return group > 0 || tiles >= 2 * kMinCut;
}

static int tile_pairs() { return std::min(std::max(1, num_sms() / 2), kMaxPairs); }

static size_t parts_layout(const BatchView& b, int D, int window, int group, void* base, ChunkParts* w) {
  *w = ChunkParts{};
  if (!may_cut(b, window, group)) return 0;
  uint8_t* at = static_cast<uint8_t*>(base);
  size_t used = 0;
  auto take = [&](size_t bytes) {
    uint8_t* r = at + used;
    used += align_up(bytes, 256);
    return r;
  };
  const size_t pairs = tile_pairs(), rows = pairs * 2 * kTileRows;
  w->rec = reinterpret_cast<int4*>(take(pairs * sizeof(int4)));
  w->ml = reinterpret_cast<float2*>(take(rows * sizeof(float2)));
  w->o = reinterpret_cast<float*>(take(rows * D * sizeof(float)));
  return used;
}

// Where keys and values are.
struct ChunkSource {
  const void* k;
  const void* v;
  int64_t kv_stride;   // packed: entries from row to row
};

template <typename T, int DP, bool PAGED, bool GROUPS>
static qcf_status tile_launch(const char* who, const ChunkSource& src, const PagedView& c, const BatchView& b, const ChunkArgs& p, const ChunkParts& w,
                              cudaStream_t st) {
  using Cfg = TileCfg<DP>;
  CUtensorMap tk, tv, tq, to, tp;
  const CUtensorMapSwizzle v_swizzle = Cfg::VCOLS == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  const uint64_t qd[3] = {static_cast<uint64_t>(p.D), static_cast<uint64_t>(p.a.Hq), static_cast<uint64_t>(b.n_rows)};
  const uint64_t qs[2] = {static_cast<uint64_t>(p.D) * 2, static_cast<uint64_t>(p.a.q_stride) * 2};
  const uint32_t qb[3] = {64, static_cast<uint32_t>(p.a.G), static_cast<uint32_t>(p.per)};
  const uint64_t os[2] = {static_cast<uint64_t>(p.D) * 2, static_cast<uint64_t>(p.a.Hq) * p.D * 2};
  bool ok = encode_tmap_3d(&tq, p.a.q, qd, qs, qb, CU_TENSOR_MAP_SWIZZLE_128B) && encode_tmap_3d(&to, p.a.o, qd, os, qb, CU_TENSOR_MAP_SWIZZLE_128B);
  if (w.rec)   // sums of the parts: rows of D columns, boxes of 128 rows and 32 columns
    ok = ok && encode_tmap_2d(&tp, w.o, p.D, static_cast<uint64_t>(tile_pairs()) * 2 * kTileRows, static_cast<uint64_t>(p.D) * 4, 32, 128,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_DATA_TYPE_FLOAT32);
  else
    tp = to;     // never used
  if (PAGED) {
    ok = ok && encode_pages(&tk, src.k, c, std::min(1 << c.page_shift, 64), 64, CU_TENSOR_MAP_SWIZZLE_128B) &&
         encode_pages(&tv, src.v, c, std::min(1 << c.page_shift, kTileKeys), Cfg::VCOLS, v_swizzle);
  } else {
    const uint64_t d[3] = {static_cast<uint64_t>(p.D), static_cast<uint64_t>(c.Hkv), static_cast<uint64_t>(b.n_rows)};
    const uint64_t s[2] = {static_cast<uint64_t>(p.D) * 2, static_cast<uint64_t>(src.kv_stride) * 2};
    const uint32_t kb[3] = {64, 1, 64}, vb[3] = {Cfg::VCOLS, 1, kTileKeys};
    ok = ok && encode_tmap_3d(&tk, src.k, d, s, kb, CU_TENSOR_MAP_SWIZZLE_128B) && encode_tmap_3d(&tv, src.v, d, s, vb, v_swizzle);
  }
  if (!ok) return set_error(QCF_ERR_CUDA, "%s: tensor map encoding failed", who);
  static PerDevice<cudaError_t> smem_attr;
  cudaError_t e = smem_attr.get(current_device(), [] {
    return cudaFuncSetAttribute(tile_attn_kernel<T, DP, PAGED, GROUPS>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM);
  });
  if (e != cudaSuccess) return cuda_error(e, who);
  {
    LaunchScope ls(KC_CHUNK_ATTN, st);
    e = launch_pdl(tile_attn_kernel<T, DP, PAGED, GROUPS>, dim3(2 * tile_pairs()), dim3(kTileThreads), Cfg::SMEM, st, tk, tv, tq, to, tp, c, b, p, w,
                   device_status_ptr());
    if (e != cudaSuccess) return cuda_error(e, who);
  }
  if (!w.rec) return QCF_OK;
  LaunchScope ls(KC_CHUNK_JOIN, st);
  e = launch_pdl(tile_join_kernel<T>, dim3(num_sms() * 4), dim3(kJoinThreads), 0, st, p, w, tile_pairs());
  return e == cudaSuccess ? QCF_OK : cuda_error(e, who);
}

template <typename T, bool PAGED>
static qcf_status tile_launch_type(const char* who, const ChunkSource& src, const PagedView& c, const BatchView& b, const ChunkArgs& p, const ChunkParts& w,
                                   cudaStream_t st) {
  if constexpr (PAGED)
    if (p.group > 0)
      return p.D <= 64 ? tile_launch<T, 64, PAGED, true>(who, src, c, b, p, w, st) : tile_launch<T, 128, PAGED, true>(who, src, c, b, p, w, st);
  return p.D <= 64 ? tile_launch<T, 64, PAGED, false>(who, src, c, b, p, w, st) : tile_launch<T, 128, PAGED, false>(who, src, c, b, p, w, st);
}

template <bool PAGED>
static qcf_status chunk_launch(const char* who, int dtype, const ChunkSource& src, const PagedView& c, const BatchView& b, ChunkArgs p, void* ws,
                               size_t ws_bytes, cudaStream_t st) {
  if (p.window >= static_cast<int64_t>(b.prefix_len) + b.max_len) p.window = 0;   // every key lies inside
  ChunkParts w;
  const size_t need = parts_layout(b, p.D, p.window, p.group, ws, &w);
  if (need > 0 && (!ws || ws_bytes < need)) return set_error(QCF_ERR_WORKSPACE, "%s: workspace %zu < %zu", who, ws_bytes, need);
  if (dtype == QCF_BF16) return tile_launch_type<__nv_bfloat16, PAGED>(who, src, c, b, p, w, st);
  return tile_launch_type<__half, PAGED>(who, src, c, b, p, w, st);
}

static qcf_status check_sizes(const char* who, const PagedView& c, const BatchView& b, int Hq) {
  if (b.n_seq > kMaxChunkSeqs) return set_error(QCF_ERR_SHAPE, "%s: n_seq=%d (at most %d)", who, b.n_seq, kMaxChunkSeqs);
  if (Hq <= 0 || Hq % c.Hkv || Hq / c.Hkv > 128) return set_error(QCF_ERR_SHAPE, "%s: Hq=%d Hkv=%d", who, Hq, c.Hkv);
  if (static_cast<int64_t>(b.n_rows) * Hq > INT32_MAX / 128)
    return set_error(QCF_ERR_SHAPE, "%s: %d rows of %d heads are too many for one call", who, b.n_rows, Hq);
  // the deal counts costs in 31 bits, with room for a share more
  const int R = 4 * (128 / (Hq / c.Hkv));
  const double blocks = std::min(static_cast<double>(b.n_seq) * ((std::min(b.max_q, b.n_rows) + R - 1) / R), static_cast<double>(b.n_rows) / R + b.n_seq);
  if (blocks * c.Hkv * (kUnitCost + kGroupCost2 * static_cast<double>(most_tiles(b))) > INT32_MAX / 2)
    return set_error(QCF_ERR_SHAPE, "%s: the bounds allow more work than one call takes", who);
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
  if (check_packed("qcf_packed_causal_attn_workspace_size", n_seq, n_rows, max_len, Hq, Hkv, D, &c, &b) != QCF_OK) return 0;
  ChunkParts w;
  return n_seq == 0 || n_rows == 0 ? 0 : parts_layout(b, D, 0, 0, nullptr, &w);
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
  const ChunkArgs p{attn_args(q, q_stride, o, lse, Hq, Hkv, scale), D, window, 128 / (Hq / Hkv), 0};
  return chunk_launch<false>(who, dtype, ChunkSource{k, v, kv_stride}, c, b, p, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

size_t qcf_paged_chunk_attn_workspace_size(const qcf_paged_kv* cache, const qcf_paged_batch* batch, int Hq) {
  const char* who = "qcf_paged_chunk_attn_workspace_size";
  PagedView c;
  BatchView b;
  if (check_paged(who, cache, batch, &c, &b) != QCF_OK || check_sizes(who, c, b, Hq) != QCF_OK) return 0;
  ChunkParts w;
  return b.n_seq == 0 || b.n_rows == 0 ? 0 : parts_layout(b, c.D, 0, group_rows(b, 0, 128 / (Hq / c.Hkv)), nullptr, &w);
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
  const int per = 128 / (Hq / c.Hkv);
  const ChunkArgs p{attn_args(q, q_stride, o, lse, Hq, c.Hkv, scale), c.D, window, per, group_rows(b, window, per)};
  return chunk_launch<true>(who, cache->dtype, ChunkSource{cache->k, cache->v, 0}, c, b, p, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
