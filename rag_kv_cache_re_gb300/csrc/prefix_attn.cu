// The shared prefix of a batch on tcgen05 tensor cores (head dims 64 and 128): its K and V are
// loaded once for every 256 score rows of a KV head (2 (128 / G) rows of the batch), and by the units
// of further rows out of L2 as far as they fit.
//
// The score rows of one KV head (rows of the batch x the G query heads that share it) are stacked
// into units of two 128-row tiles, a and b, which share every K and V tile of 128 keys.  The tiles
// of all (row block, KV head) units are dealt out evenly: CTA i takes tiles [i share, (i + 1)
// share) of the whole sequence of units, so the SMs finish together whatever the batch, and a CTA
// leaves one part for each unit it touched (two or three at most when share is large).
//
// Twelve warps:
//   warp 0      K producer: pages to shared memory by tiled TMA, one box per page and 64 columns,
//               page ids by lane; also Q, both row tiles of a unit
//   warp 2      V producer, the same; rows behind the prefix in its last page are zeroed, since a
//               free slot may hold NaN and 0 x NaN is NaN
//   warps 1, 3  one thread each issues the products of row tile x = a, b: P_x V, then S_x = Q_x K^T
//               of the next key tile, while the other tile is in its softmax.  A thread spends
//               about 72 cycles on a 64-cycle product and 60 to 160 on each barrier, so one thread
//               for both tiles was slower than the tensor pipe.  The two take turns: left free,
//               their products mix, both tiles finish together and then both wait for their softmax
//   warps 4-7   softmax of a, warps 8-11 of b: thread = score row; maximum, powers of two and sum
//               in fp32, the weights back to tensor memory over the scores they came from (they
//               meet V in the cache's 16-bit type, the MMA's), the output rescaled in tensor
//               memory only when a row's maximum grows by more than 2^8
// Tensor memory columns: S_a 0, S_b 128 (128 each; the weights take the first 64 of each), O_a
// 256, O_b 256 + D.  A commit covers every product issued before it, so a full S_x(i + 1) also
// means that P_x(i) V has been added: no barrier of its own for the output.
//
// Bound: HBM below about 285 score rows per KV head, the tensor pipe above.  131072 keys of 8 KV heads
// against 256 score rows each: 99 us, 5.4 TB/s and 1.39 PFLOP/s at once; 16384 keys against 1564: 80 us,
// 1.31 PFLOP/s.  A pair of 128 x 128 tiles takes 2860 to 3030 cycles, 2048 of them products: the S
// products read both operands from shared memory at its full rate.  ptxas, which plans for 168 registers in every
// warp, spills 12 bytes a thread.  At head dim 64, with half the products to a tile and the same
// softmax, the call with 131072 keys and 256 score rows a KV head takes 99 us (116 at 128; floor 41).
#include <algorithm>

#include "paged_attn.cuh"

namespace qcf {

constexpr int kPreKeys = 128;
constexpr int kPreThreads = 384;
constexpr int kPreBox = kPreKeys * 128;   // bytes of 64 columns of 128 keys (or score rows)

template <int D>
struct PreCfg {
  static constexpr int BOXES = D / 64;
  static constexpr int TILE = BOXES * kPreBox;               // a K, V or Q tile
  static constexpr int K_STAGES = D == 128 ? 3 : 5;          // K runs a tile ahead of V
  static constexpr int V_STAGES = D == 128 ? 2 : 5;
  static constexpr int SMEM = (2 + K_STAGES + V_STAGES) * TILE + 512 + 1024;
};

// Instruction descriptor of kind::f16 with both operands of type T (see idesc_bf16_f32).
template <typename T>
constexpr uint32_t idesc_16(int M, int N, bool b_mn_major) {
  return std::is_same<T, __half>::value ? idesc_bf16_f32(M, N, b_mn_major) & ~((1u << 7) | (1u << 10))
                                        : idesc_bf16_f32(M, N, b_mn_major);
}

// One CTA's share of one unit.
struct Segment {
  int g, row0, nb, t0, nt, part;   // KV head, first row of tile a, row tiles in use, key tiles, part slot
};
struct Segments {
  int cur, end, cta;
  const SharedPlan& p;
  int n_rows;
  __device__ Segments(const SharedPlan& plan, int n_rows_, int total)
      : cta(static_cast<int>(blockIdx.x)), p(plan), n_rows(n_rows_) {
    if (p.pre_even) {   // CTA = (part, unit): the units' same parts start together
      const int units = total / p.pre_tiles, unit = cta % units, part = cta / units;
      cur = unit * p.pre_tiles + static_cast<int>(static_cast<int64_t>(part) * p.pre_tiles / p.pre_parts);
      end = unit * p.pre_tiles + static_cast<int>(static_cast<int64_t>(part + 1) * p.pre_tiles / p.pre_parts);
      cta = part;
    } else {
      cur = cta * p.pre_share;
      end = min(total, cur + p.pre_share);
    }
  }
  __device__ bool next(Segment& s) {
    if (cur >= end) return false;
    const int unit = cur / p.pre_tiles;
    s.t0 = cur - unit * p.pre_tiles;
    s.nt = min(p.pre_tiles - s.t0, end - cur);
    s.g = unit / p.pre_row_blocks;
    s.row0 = (unit - s.g * p.pre_row_blocks) * p.pre_rows;
    s.nb = s.row0 + p.pre_rows / 2 < n_rows ? 2 : 1;
    s.part = p.pre_even ? cta : cta - unit * p.pre_tiles / p.pre_share;
    cur += s.nt;
    return true;
  }
};

__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, const void* smem_src, int x, int y, int z, int w) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];"
               ::"l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(smem_src)), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}
// The shared memory of this thread's bulk stores has been read.
__device__ __forceinline__ void bulk_wait_read0() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

template <typename T, int D>
__global__ void __launch_bounds__(kPreThreads, 1)
    prefix_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmO, const PagedView c, const BatchView b, const AttnArgs a,
                       const SharedPlan p, const Workspace ws, int total, unsigned int* status) {
  using Cfg = PreCfg<D>;
  constexpr int KST = Cfg::K_STAGES, VST = Cfg::V_STAGES;
  constexpr unsigned kAll = 0xffffffffu;
  // Launched while the stream kernel runs, on whose results nothing here depends.  What this kernel
  // does depend on (queries, pages, the join of the call before, which reads the parts that are
  // written here) has ended before the stream began, for the stream is launched without the programmatic
  // attribute.  The join waits for this kernel alone, so this one ends after the stream has (its
  // pdl_wait).
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmO);
  }
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* qbuf = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  uint8_t* kbuf = qbuf + 2 * Cfg::TILE;
  uint8_t* vbuf = kbuf + KST * Cfg::TILE;
  uint64_t* k_full = reinterpret_cast<uint64_t*>(vbuf + VST * Cfg::TILE);
  uint64_t* k_empty = k_full + KST;
  uint64_t* v_full = k_empty + KST;
  uint64_t* v_empty = v_full + VST;
  uint64_t* s_full = v_empty + VST;    // [a, b]
  uint64_t* p_ready = s_full + 2;     // [a, b][first, last 64 keys]
  uint64_t* o_done = p_ready + 4;     // [a, b]
  uint64_t* q_full = o_done + 2;
  uint64_t* q_empty = q_full + 1;
  uint64_t* v_tail = q_empty + 1;
  uint64_t* mma_end = v_tail + 1;     // [a, b]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_end + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < KST; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 2);
    }
    for (int s = 0; s < VST; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 2);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&s_full[x], 1);
      mbar_init(&p_ready[2 * x], 5);
      mbar_init(&p_ready[2 * x + 1], 4);
      mbar_init(&o_done[x], 1);
      mbar_init(&mma_end[x], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 4);   // both issuers' products have read Q, both tiles' sums have left through its memory
    mbar_init(v_tail, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Segments segs(p, b.n_rows, total);
  Segment s;

  if (warp < 4) {
    // 104 x 128 + 200 x 256 threads: the 168 x 384 registers of the launch
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == 0 || warp == 2) {
      // ---- K and V producers
      const bool is_k = warp == 0;
      const CUtensorMap* map = is_k ? &tmK : &tmV;
      uint8_t* ring = is_k ? kbuf : vbuf;
      uint64_t* full = is_k ? k_full : v_full;
      uint64_t* empty = is_k ? k_empty : v_empty;
      const int ST = is_k ? KST : VST;
      const int ps = min(1 << c.page_shift, kPreKeys), boxes = kPreKeys / ps;   // rows of a box, pages of a tile
      // this lane's page of key tile t: its id, n_pages (which reads as zeros) where there is none
      auto page_of = [&](int t) {
        const int key = t * kPreKeys + lane * ps;
        if (lane >= boxes || key >= b.prefix_len) return c.n_pages;
        const int id = b.prefix_pages[key >> c.page_shift];
        if (id >= 0 && id < c.n_pages) return id;
        flag_status(status, QCF_DEV_BAD_INDEX);
        return c.n_pages;
      };
      int n = 0, tails = 0, k = 0;   // tiles, tail tiles, units of Q so far
      bool ok = true;
      while (ok && segs.next(s)) {
        int id = page_of(s.t0);
        for (int i = 0; i < s.nt; ++i, ++n) {
          const int st = n % ST, t = s.t0 + i;
          const int next_id = i + 1 < s.nt ? page_of(t + 1) : 0;
          if (!__all_sync(kAll, mbar_wait(&empty[st], ((n / ST) & 1) ^ 1u))) {
            ok = false;
            break;
          }
          const int valid = b.prefix_len - t * kPreKeys;   // keys of this tile (at least one)
          const int stale = valid < kPreKeys ? min(kPreKeys, (valid + ps - 1) / ps * ps) : valid;
          const bool tail = !is_k && stale > valid;        // a page of the tile ends behind the prefix
          uint64_t* bar = tail ? v_tail : &full[st];
          uint8_t* dst = ring + st * Cfg::TILE;
          if (lane == 0) mbar_arrive_expect_tx(bar, Cfg::TILE);
          __syncwarp();
          if (lane < boxes) {
#pragma unroll
            for (int h = 0; h < Cfg::BOXES; ++h)
              tma_load_4d(dst + h * kPreBox + lane * ps * 128, map, bar, h * 64, (t * kPreKeys) & ((1 << c.page_shift) - 1), s.g,
                          id);
          }
          id = next_id;
          if (is_k && i == 0) {   // the unit's Q; rows behind the batch are zeros
            if (!__all_sync(kAll, mbar_wait(q_empty, (k & 1) ^ 1u))) {
              ok = false;
              break;
            }
            const int per = 128 / a.G;
            if (lane == 0) mbar_arrive_expect_tx(q_full, s.nb * Cfg::BOXES * per * a.G * 128);
            __syncwarp();
            if (lane < s.nb * Cfg::BOXES)
              tma_load_3d(qbuf + lane * kPreBox, &tmQ, q_full, lane % Cfg::BOXES * 64, s.g * a.G, s.row0 + lane / Cfg::BOXES * per);
            ++k;
          }
          if (tail) {
            if (!__all_sync(kAll, mbar_wait(v_tail, tails++ & 1))) {
              ok = false;
              break;
            }
            for (int e = lane; e < (stale - valid) * 8 * Cfg::BOXES; e += 32) {
              const int h = e / ((stale - valid) * 8), f = e - h * (stale - valid) * 8;
              *reinterpret_cast<uint4*>(dst + h * kPreBox + valid * 128 + f * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[st]);
          }
        }
      }
      if (!ok && lane == 0) flag_status(status, QCF_DEV_TIMEOUT);
      // no copy of this warp is in flight when the CTA ends
      for (int e = max(0, n - ST); e < n; ++e)
        if (!mbar_wait(&full[e % ST], (e / ST) & 1) && lane == 0) flag_status(status, QCF_DEV_TIMEOUT);
      if (k > 0 && !mbar_wait(q_full, (k - 1) & 1) && lane == 0) flag_status(status, QCF_DEV_TIMEOUT);
    } else if (lane == 0) {
      // ---- MMA issuer of row tile x
      const int x = warp >> 1;
      constexpr uint32_t idesc_s = idesc_16<T>(128, kPreKeys, false);
      constexpr uint32_t idesc_o = idesc_16<T>(128, D, true);
      int n = 0, k = 0;    // key tiles, segments so far
      uint32_t used = 0;   // weight tiles taken so far
      bool ok = true;
      // a descriptor's low 14 bits are the address in 16-byte units: steps inside a tile are added to it
      const uint64_t q_desc = sdesc_kmajor_sw128(smem_u32(qbuf + x * Cfg::TILE));
      const uint64_t k_desc = sdesc_kmajor_sw128(smem_u32(kbuf)), v_desc = sdesc_mnmajor_sw128(smem_u32(vbuf), kPreBox);
      // The turn: the barrier of a tile's first weights also counts one arrival of the other
      // issuer, made four products (256 cycles) before the end of its block, which covers what
      // this thread then takes to see it.
      auto pass = [&](bool due) {
        if (due) mbar_arrive(&p_ready[2 * (1 - x)]);
      };
      auto scores = [&](int tile, bool due) {   // S_x = Q_x K^T
        const uint64_t kd = k_desc + tile % KST * (Cfg::TILE >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          if (kk == D / 16 - 4) pass(due);
          const uint64_t at = ((kk >> 2) * kPreBox + (kk & 3) * 32) >> 4;
          umma_f16(tmem + x * 128, q_desc + at, kd + at, idesc_s, kk > 0 ? 1u : 0u);
        }
        umma_commit(&s_full[x]);
        umma_commit(&k_empty[tile % KST]);
      };
      auto wait_k = [&](int tile) { return mbar_wait(&k_full[tile % KST], (tile / KST) & 1); };
      for (; ok && segs.next(s); ++k) {
        if (x >= s.nb) {   // nothing in tile b: hand on what it would have read (every phase of a barrier is waited for)
          if (!(ok = mbar_wait(q_full, k & 1))) break;
          mbar_arrive(q_empty);
          mbar_arrive(q_empty);   // for the softmax of b too
          for (int i = 0; i < s.nt; ++i, ++n) {
            if (!(ok = wait_k(n))) break;
            mbar_arrive(&k_empty[n % KST]);
            if (!(ok = mbar_wait(&v_full[n % VST], (n / VST) & 1))) break;
            mbar_arrive(&v_empty[n % VST]);
          }
          continue;
        }
        if (!(ok = mbar_wait(q_full, k & 1) && wait_k(n))) break;
        tc_fence_after();
        scores(n, false);
        for (int i = 0; i < s.nt; ++i, ++n) {
          const bool more = i + 1 < s.nt;
          if (!(ok = mbar_wait(&v_full[n % VST], (n / VST) & 1) && (!more || wait_k(n + 1)))) break;
          const uint64_t vd = v_desc + n % VST * (Cfg::TILE >> 4);
          auto weigh = [&](int half) {   // O_x += P_x V over 64 keys
            tc_fence_after();
#pragma unroll
            for (int kk = half * (kPreKeys / 32); kk < (half + 1) * (kPreKeys / 32); ++kk)
              umma_f16_ts(tmem + 256 + x * D, tmem + x * 128 + kk * 8, vd + kk * (2048 >> 4), idesc_o,
                          (i > 0 || kk > 0) ? 1u : 0u);
          };
          // a alone, or first of the unit, gives itself the turn; b's last block passes none
          if (x == 0 && (s.nb == 1 || i == 0)) mbar_arrive(&p_ready[0]);
          const bool due = s.nb == 2 && (x == 0 || more);
          if (!(ok = mbar_wait(&p_ready[2 * x], used & 1))) break;
          weigh(0);
          if (!(ok = mbar_wait(&p_ready[2 * x + 1], used & 1))) break;
          weigh(1);
          ++used;
          if (more) {
            scores(n + 1, due);
          } else {
            pass(due);
            umma_commit(&o_done[x]);
          }
          umma_commit(&v_empty[n % VST]);   // after the scores: a commit costs this thread more than a product
        }
        umma_commit(q_empty);
      }
      if (!ok) flag_status(status, QCF_DEV_TIMEOUT);
      umma_commit(&mma_end[x]);   // nothing runs on tensor memory once it is freed
      if (!mbar_wait(&mma_end[x], 0)) flag_status(status, QCF_DEV_TIMEOUT);
    }
  } else {
    // ---- softmax: thread = score row of tile x
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    const int x = (warp - 4) >> 2, quarter = warp & 3;
    const int rho = quarter * 32 + lane, per = 128 / a.G, pl = rho / a.G, h = rho - pl * a.G;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_tm = tmem + lane_base + x * 128, o_tm = tmem + lane_base + 256 + x * D;
    auto page_bad = [&](int t) {   // the page of this lane's 8 keys of tile t lies outside the cache
      const int key = t * kPreKeys + lane * 8;
      if (lane >= kPreKeys / 8 || key >= b.prefix_len) return false;
      const int id = b.prefix_pages[key >> c.page_shift];
      return id < 0 || id >= c.n_pages;
    };
    uint32_t seen = 0, ends = 0;
    bool ok = true;   // a warp whose wait ran out still meets the others at the tile's barriers
    while (segs.next(s)) {
      if (x >= s.nb) continue;
      const int row = s.row0 + x * per + pl;
      float m = -INFINITY, l = 0.f;
      bool bad = page_bad(s.t0);
      for (int i = 0; ok && i < s.nt; ++i) {
        const int t = s.t0 + i;
        const unsigned bad8 = __ballot_sync(kAll, bad);
        bad = i + 1 < s.nt && page_bad(t + 1);
        if (!__all_sync(kAll, mbar_wait(&s_full[x], seen++ & 1))) {
          ok = false;
          break;
        }
        tc_fence_after();
        float sv[kPreKeys];
        tmem_ld128(s_tm, sv);
        const int valid = b.prefix_len - t * kPreKeys;
        if (valid < kPreKeys) {
#pragma unroll
          for (int j = 0; j < kPreKeys; ++j)
            if (j >= valid) sv[j] = -INFINITY;
        }
        if (bad8) {
#pragma unroll
          for (int j = 0; j < kPreKeys; ++j)
            if (bad8 >> (j / 8) & 1) sv[j] = -INFINITY;
        }
        // 64 weights from the logits; they leave in two halves, so that P V of the first 64 keys runs
        // under the powers of the others
        const Pair scale2 = make_pair2(a.scale_log2, a.scale_log2);
        Pair sum[2];
        uint32_t pk[32];
        auto weights = [&](int half, float base) {
          const Pair nm2 = make_pair2(-base, -base);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int j = half * 64 + 2 * e;
            float p0, p1;
            split(fma2(make_pair2(sv[j], sv[j + 1]), scale2, nm2), p0, p1);
            p0 = fast_exp2(p0);
            p1 = fast_exp2(p1);
            sum[e & 1] = add2(sum[e & 1], make_pair2(p0, p1));
            pk[e] = pack2<T>(p0, p1);
          }
        };
        // The first half is weighed with the maximum so far, the tile's own found meanwhile (the
        // special-function unit paces the powers, the comparisons fill its gaps): the maximum
        // moves only by more than 2^8, so after a unit's first tiles it nearly always stands.
        sum[0] = sum[1] = make_pair2(0.f, 0.f);
        weights(0, m == -INFINITY ? 0.f : m);
        float mx[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
        for (int j = 4; j < kPreKeys - 4; j += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], sv[j + e], sv[j + 4 + e]);
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], sv[kPreKeys - 4 + e]);
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
        const bool grow = top > m + (8.0f + kWeightLift<T>);
        if (__any_sync(kAll, grow)) {
          const float m_new = grow ? top - kWeightLift<T> : m;
          if (i > 0) {   // the full S of this tile says that every earlier product has been added to O
            const float f = m == -INFINITY ? 0.f : fast_exp2(m - m_new);
#pragma unroll 1
            for (int cc = 0; cc < D / 32; ++cc) {
              float ov[32];
              tmem_ld32(o_tm + cc * 32, ov);
#pragma unroll
              for (int e = 0; e < 32; ++e) ov[e] *= f;
              tmem_st32(o_tm + cc * 32, ov);
            }
            l *= f;
          }
          m = m_new;
          sum[0] = sum[1] = make_pair2(0.f, 0.f);
          weights(0, m == -INFINITY ? 0.f : m);
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (half == 1) weights(1, m == -INFINITY ? 0.f : m);
          tmem_st32u(s_tm + half * 32, pk);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_ready[2 * x + half]);
        }
        float l0, l1;
        split(add2(sum[0], sum[1]), l0, l1);
        l += l0 + l1;
      }
      ok = ok && __all_sync(kAll, mbar_wait(&o_done[x], ends++ & 1));
      tc_fence_after();
      // The sums leave through the tile's Q memory (its products are done: O is), 32 columns a box, by
      // tiled TMA stores of whole lines, rows behind the batch cut off; written row by row from the
      // threads that hold them they took 7 us.
      if (pl < per && row < b.n_rows)
        ws.tc_ml[(static_cast<int64_t>(s.part) * b.n_rows + row) * a.Hq + s.g * a.G + h] = make_float2(m, l);
      uint8_t* stage = qbuf + x * Cfg::TILE;
#pragma unroll 1
      for (int c0 = 0; c0 < D / 32; c0 += Cfg::BOXES) {
        if (c0 > 0) {
          if (rho == 0) bulk_wait_read0();
          bar_sync(1 + x, 128);
        }
#pragma unroll
        for (int cc = 0; cc < Cfg::BOXES; ++cc) {
          float ov[32];
          tmem_ld32(o_tm + (c0 + cc) * 32, ov);
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(stage + cc * kPreBox + sw128_off(rho, e / 4)) = make_float4(ov[e], ov[e + 1], ov[e + 2], ov[e + 3]);
        }
        fence_proxy_async_smem();
        bar_sync(1 + x, 128);
        if (rho == 0) {
#pragma unroll
          for (int cc = 0; cc < Cfg::BOXES; ++cc)
            tma_store_4d(&tmO, stage + cc * kPreBox, (c0 + cc) * 32, s.g * a.G, s.row0 + x * per, s.part);
          bulk_commit_group();
        }
      }
      tc_fence_before();
      if (rho == 0) {
        bulk_wait_read0();
        mbar_arrive(q_empty);
      }
    }
    if (rho == 0) bulk_wait_group0();   // the stores are done, not only read, before this kernel counts as complete
    if (!ok && lane == 0) flag_status(status, QCF_DEV_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  pdl_wait();
}

template <typename T, int D>
static qcf_status prefix_tc_type(const qcf_paged_kv* cache, const PagedView& c, const BatchView& b, const AttnArgs& a,
                                 const SharedPlan& p, const Workspace& w, cudaStream_t st) {
  using Cfg = PreCfg<D>;
  CUtensorMap tk, tv, tq, to;
  const int rows = std::min(1 << c.page_shift, kPreKeys);
  const uint64_t qd[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(a.Hq), static_cast<uint64_t>(b.n_rows)};
  const uint64_t qs[2] = {static_cast<uint64_t>(D) * 2, static_cast<uint64_t>(a.q_stride) * 2};
  const uint64_t od[4] = {static_cast<uint64_t>(D), static_cast<uint64_t>(a.Hq), static_cast<uint64_t>(b.n_rows),
                          static_cast<uint64_t>(p.pre_parts)};
  const uint64_t os[3] = {static_cast<uint64_t>(D) * 4, static_cast<uint64_t>(a.Hq) * D * 4,
                          static_cast<uint64_t>(b.n_rows) * a.Hq * D * 4};
  const uint32_t ob[4] = {32, static_cast<uint32_t>(a.G), static_cast<uint32_t>(128 / a.G), 1};
  const uint32_t qb[3] = {64, static_cast<uint32_t>(a.G), static_cast<uint32_t>(128 / a.G)};
  if (!encode_pages(&tk, cache->k, c, rows, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_pages(&tv, cache->v, c, rows, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_tmap_3d(&tq, a.q, qd, qs, qb, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_tmap_4d(&to, w.tc_o, od, os, ob, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_DATA_TYPE_FLOAT32))
    return set_error(QCF_ERR_CUDA, "qcf_shared_prefix_attn: tensor map encoding failed");
  static PerDevice<cudaError_t> smem_attr;
  const cudaError_t attr = smem_attr.get(current_device(), [] {
    return cudaFuncSetAttribute(prefix_attn_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM);
  });
  if (attr != cudaSuccess) return cuda_error(attr, "qcf_shared_prefix_attn: smem attribute");
  LaunchScope ls(KC_PREFIX_ATTN, st);
  const int total = p.pre_tiles * p.pre_row_blocks * c.Hkv;
  const cudaError_t e = launch_pdl(prefix_attn_kernel<T, D>, dim3(p.pre_ctas), dim3(kPreThreads), Cfg::SMEM, st, tk, tv, tq, to, c, b, a,
                                   p, w, total, device_status_ptr());
  return e == cudaSuccess ? QCF_OK : cuda_error(e, "qcf_shared_prefix_attn: prefix launch");
}

qcf_status prefix_tc_launch(const qcf_paged_kv* cache, const PagedView& c, const BatchView& b, const AttnArgs& a,
                            const SharedPlan& p, const Workspace& w, cudaStream_t st) {
  if (cache->dtype == QCF_BF16)
    return c.D == 128 ? prefix_tc_type<__nv_bfloat16, 128>(cache, c, b, a, p, w, st)
                      : prefix_tc_type<__nv_bfloat16, 64>(cache, c, b, a, p, w, st);
  return c.D == 128 ? prefix_tc_type<__half, 128>(cache, c, b, a, p, w, st)
                    : prefix_tc_type<__half, 64>(cache, c, b, a, p, w, st);
}

}  // namespace qcf
