// Attention of a batch of sequences over a shared prefix and their own tokens, both in pages.
//
// With logits x_j = scale q.K_j, any set of keys P is summed up by M = max x_j, L = sum 2^(x_j - M)
// (x in powers of two) and O = sum 2^(x_j - M) V_j; two sets join by scaling each with
// 2^(M - max M).  The keys of a row are split into such parts: chunks of the prefix, scored for
// all rows of the batch together so that its K and V are read once, and chunks of the sequence's
// own tokens.  A last kernel joins the parts of each row.
#include <algorithm>
#include <cmath>

#include "paged_attn.cuh"

namespace qcf {

// ------------------------------------------------------------------ parts on warp tensor cores
//
// A unit is up to 64 score rows (new rows x the G query heads of one KV head) of one sequence
// against a chunk of its own keys, or up to 64 rows of the whole batch against a chunk of the
// prefix.  Four warps stream tiles of 64 keys through a ring in shared memory, 16 keys of a tile
// each, with 16-byte asynchronous copies whose addresses come from the page table (keys behind
// the chunk and keys of bad pages arrive as zeros, so nothing a free slot holds is ever
// multiplied).  Up to 16 score rows (single tokens): the rows fit one MMA tile, every warp keeps
// all of them and scores the 16 keys it copied itself, so the warps run free of each other and
// join at the end.  More rows: 16 to a warp, and every warp scores the whole tile.
// Single tokens are bound by the K and V bytes: the ring keeps 64 KB (D = 128) in flight per CTA.
constexpr int kOwnWarps = 4;
constexpr int kOwnTile = 16 * kOwnWarps;   // keys
constexpr int kOwnRows = 64;               // score rows of a unit

template <int D>
struct OwnCfg {
  static constexpr int STAGES = D == 128 ? 3 : 4;
  static constexpr int GROUP = 16 * D * 2;                  // bytes of 16 keys (or values)
  static constexpr int STAGE = 2 * kOwnWarps * GROUP;       // K groups, then V groups
  static constexpr int MERGE = kOwnWarps * 16 * D * 4 + kOwnWarps * 16 * 8;
  static constexpr int SMEM = STAGES * STAGE > MERGE ? STAGES * STAGE : MERGE;
  static constexpr int MIN_CTAS = D == 128 ? 2 : 3;
};

// Byte offset of 8 entries at column col of a key in a group; 16-byte pieces are permuted by the
// key so that eight keys' pieces of one column fall into different banks.
template <int D>
__device__ __forceinline__ uint32_t group_off(int key, int col) {
  if constexpr (D >= 64)
    return static_cast<uint32_t>(key * (D * 2) + (((col >> 3) ^ (key & 7)) << 4));
  else
    return static_cast<uint32_t>(key * (D * 2) + (((col >> 3) ^ ((key >> 2) & 1)) << 4));
}

template <typename T, int D>
__global__ void __launch_bounds__(kOwnWarps * 32, OwnCfg<D>::MIN_CTAS)
    own_attn_kernel(const PagedView c, const BatchView b, const AttnArgs a, const SharedPlan p, const Parts parts,
                    int pre_units, unsigned int* status) {
  using Cfg = OwnCfg<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- the unit: rows rho0 .. rho0 + rows, keys [k0, k1) of `pages`, part slot `part`
  int u = static_cast<int>(blockIdx.x);
  const bool pre = u < pre_units;
  if (!pre) u -= pre_units;
  const int g = u % c.Hkv;
  u /= c.Hkv;
  int rho0, row0, n_rho, part, k0, k1, last0;   // last0: the last key that score row rho = 0 sees
  const int32_t* pages;
  bool only = false;                             // the row's only part: written to o at once
  if (pre) {
    const int chunk = u % p.pre_parts;
    rho0 = u / p.pre_parts * kOwnRows;
    row0 = 0;
    n_rho = b.n_rows * a.G;
    part = chunk;
    k0 = chunk * p.pre_chunk;
    k1 = min(b.prefix_len, k0 + p.pre_chunk);
    last0 = b.prefix_len;                        // no row's limit
    pages = b.prefix_pages;
  } else {
    const int chunk = u % p.own_parts;
    u /= p.own_parts;
    rho0 = u % p.own_row_blocks * kOwnRows;
    const int seq = u / p.own_row_blocks;
    const SeqSpan s = seq_span(b, seq);
    if (s.bad && threadIdx.x == 0 && g == 0 && chunk == 0 && rho0 == 0) flag_status(status, QCF_DEV_BAD_INDEX);
    row0 = s.row0;
    n_rho = s.nq * a.G;
    part = p.pre_parts + chunk;
    k0 = chunk * p.own_chunk;
    k1 = min(s.len, k0 + p.own_chunk);
    last0 = s.len - s.nq;
    pages = b.page_table + static_cast<int64_t>(seq) * b.table_stride;
    only = p.pre_parts == 0 && s.len <= p.own_chunk;
    if (k0 >= s.len) return;                     // not a part of this sequence
  }
  const int rows = min(kOwnRows, n_rho - rho0);
  if (rows <= 0) return;
  const int reach = pre ? k1 : last0 + (rho0 + rows - 1) / a.G + 1;   // keys behind it are seen by no row
  k1 = min(k1, reach);
  const bool by_keys = rows <= 16;               // warps split the keys, not the rows
  const int n_tiles = k1 > k0 ? (k1 - k0 + kOwnTile - 1) / kOwnTile : 0;

  // ---- this thread's score rows: r_lo = (lane / 4), r_hi = r_lo + 8 of the warp's 16
  const int w_rho = rho0 + (by_keys ? 0 : warp * 16);
  const int lo = w_rho + (lane >> 2), hi = lo + 8, end = rho0 + rows;
  const int qc = (lane & 3) * 2;
  auto q_row = [&](int rho) {
    return static_cast<const T*>(a.q) + static_cast<int64_t>(row0 + rho / a.G) * a.q_stride +
           static_cast<int64_t>(g * a.G + rho % a.G) * D;
  };
  uint32_t qf[D / 16][4];
  {
    const T* ql = lo < end ? q_row(lo) : nullptr;
    const T* qh = hi < end ? q_row(hi) : nullptr;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      qf[ks][0] = ql ? *reinterpret_cast<const uint32_t*>(ql + ks * 16 + qc) : 0u;
      qf[ks][1] = qh ? *reinterpret_cast<const uint32_t*>(qh + ks * 16 + qc) : 0u;
      qf[ks][2] = ql ? *reinterpret_cast<const uint32_t*>(ql + ks * 16 + qc + 8) : 0u;
      qf[ks][3] = qh ? *reinterpret_cast<const uint32_t*>(qh + ks * 16 + qc + 8) : 0u;
    }
  }
  const int lim_lo = pre ? last0 : last0 + lo / a.G, lim_hi = pre ? last0 : last0 + hi / a.G;
  const int lim_min = pre ? last0 : last0 + w_rho / a.G;   // every row of the warp sees the keys up to here

  // ---- copies: tile t, this warp's 16 keys.  The page ids of the warp's next 32 tiles sit in the
  // lanes (two ids where a page holds 8 keys).
  const uint32_t ring = smem_u32(smem);
  const int ps = 1 << c.page_shift;
  const T* Kg = static_cast<const T*>(a.k) + static_cast<int64_t>(g) * c.head_stride;
  const T* Vg = static_cast<const T*>(a.v) + static_cast<int64_t>(g) * c.head_stride;
  auto ids_of = [&](int t, int which) {          // the lane's tile t + lane; -1 for a page outside the cache
    const int key = k0 + (t + lane) * kOwnTile + warp * 16 + which * 8;
    if (key >= k1) return -2;                    // behind the chunk: nothing to read
    const int id = pages[key >> c.page_shift];
    if (id >= 0 && id < c.n_pages) return id;
    flag_status(status, QCF_DEV_BAD_INDEX);
    return -1;
  };
  int id0 = -2, id1 = -2;
  auto copy_tile = [&](int t) {
    if ((t & 31) == 0) {
      id0 = ids_of(t, 0);
      if (ps == 8) id1 = ids_of(t, 1);
    }
    const int i0 = __shfl_sync(0xffffffffu, id0, t & 31);
    const int i1 = ps == 8 ? __shfl_sync(0xffffffffu, id1, t & 31) : i0;
    const int kb = k0 + t * kOwnTile + warp * 16;
    const uint32_t dst = ring + (t % Cfg::STAGES) * Cfg::STAGE + warp * Cfg::GROUP;
    constexpr int PIECES = D / 8, STEP = 32 / PIECES > 0 ? 32 / PIECES : 1;   // keys per warp-wide copy
    const int pc = lane % PIECES;
#pragma unroll
    for (int i = 0; i < 16 / STEP; ++i) {
      const int key = i * STEP + lane / PIECES;
      const int id = key < 8 ? i0 : i1;
      const bool take = kb + key < k1 && id >= 0;
      const int64_t off = take ? id * c.page_stride + ((kb + key) & (ps - 1)) * c.row_stride + pc * 8 : 0;
      const uint32_t at = dst + group_off<D>(key, pc * 8);
      cp_async16(at, Kg + off, take);
      cp_async16(at + kOwnWarps * Cfg::GROUP, Vg + off, take);
    }
  };
  // bad pages inside the group of 16 keys at kb: bit 0 the first 8 keys, bit 1 the others
  auto bad_of = [&](int kb) {
    unsigned bad = 0;
#pragma unroll
    for (int half = 0; half < 2; ++half)
      if (kb + half * 8 < k1) {
        const int id = pages[(kb + half * 8) >> c.page_shift];
        if (id < 0 || id >= c.n_pages) bad |= 1u << half;
      }
    return bad;
  };

  float m_lo = -INFINITY, m_hi = -INFINITY, l_lo = 0.f, l_hi = 0.f;
  float acc[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  const int mi = lane >> 3, mr = lane & 7;

  // 16 keys at kb, in shared memory at kaddr and vaddr
  auto score_group = [&](uint32_t kaddr, uint32_t vaddr, int kb) {
    float sc[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.f;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      uint32_t b0, b1, b2, b3;
      ldsm_x4(kaddr + group_off<D>((mi >> 1) * 8 + mr, ks * 16 + (mi & 1) * 8), b0, b1, b2, b3);
      mma_16816<T>(sc[0], qf[ks], b0, b1);
      mma_16816<T>(sc[1], qf[ks], b2, b3);
    }
    const unsigned bad = bad_of(kb);
    const bool whole = kb + 15 < k1 && kb + 15 <= lim_min && bad == 0;
    float top_lo = -INFINITY, top_hi = -INFINITY;
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x = sc[nt][e] * a.scale_log2;
        if (!whole) {
          const int key = kb + nt * 8 + qc + (e & 1);
          if (key >= k1 || key > (e < 2 ? lim_lo : lim_hi) || (bad >> nt & 1)) x = -INFINITY;
        }
        sc[nt][e] = x;
        if (e < 2) top_lo = fmaxf(top_lo, x); else top_hi = fmaxf(top_hi, x);
      }
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
      top_lo = fmaxf(top_lo, __shfl_xor_sync(0xffffffffu, top_lo, o));
      top_hi = fmaxf(top_hi, __shfl_xor_sync(0xffffffffu, top_hi, o));
    }
    // the maximum moves only when it grows by more than 2^8: the weights then stay below 2^8
    // (exact in fp32 sums, half a step in 16 bits wherever they lie) and most groups rescale nothing
    if (__any_sync(0xffffffffu, top_lo > m_lo + 8.f || top_hi > m_hi + 8.f)) {
      const float n_lo = fmaxf(m_lo, top_lo), n_hi = fmaxf(m_hi, top_hi);
      const float f_lo = m_lo == -INFINITY ? 0.f : exp2f(m_lo - n_lo), f_hi = m_hi == -INFINITY ? 0.f : exp2f(m_hi - n_hi);
      m_lo = n_lo;
      m_hi = n_hi;
      l_lo *= f_lo;
      l_hi *= f_hi;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        acc[i][0] *= f_lo;
        acc[i][1] *= f_lo;
        acc[i][2] *= f_hi;
        acc[i][3] *= f_hi;
      }
    }
    const float b_lo = m_lo == -INFINITY ? 0.f : m_lo, b_hi = m_hi == -INFINITY ? 0.f : m_hi;
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      sc[nt][0] = exp2f(sc[nt][0] - b_lo);
      sc[nt][1] = exp2f(sc[nt][1] - b_lo);
      sc[nt][2] = exp2f(sc[nt][2] - b_hi);
      sc[nt][3] = exp2f(sc[nt][3] - b_hi);
      l_lo += sc[nt][0] + sc[nt][1];
      l_hi += sc[nt][2] + sc[nt][3];
    }
    // the weights meet the values in the cache's 16-bit type (the MMA's); their sum stays fp32
    const uint32_t pa[4] = {pack2<T>(sc[0][0], sc[0][1]), pack2<T>(sc[0][2], sc[0][3]), pack2<T>(sc[1][0], sc[1][1]),
                            pack2<T>(sc[1][2], sc[1][3])};
#pragma unroll
    for (int dp = 0; dp < D / 16; ++dp) {
      uint32_t b0, b1, b2, b3;
      ldsm_x4_t(vaddr + group_off<D>((mi & 1) * 8 + mr, dp * 16 + (mi >> 1) * 8), b0, b1, b2, b3);
      mma_16816<T>(acc[2 * dp], pa, b0, b1);
      mma_16816<T>(acc[2 * dp + 1], pa, b2, b3);
    }
  };

#pragma unroll
  for (int t = 0; t < Cfg::STAGES - 1; ++t) {
    if (t < n_tiles) copy_tile(t);
    cp_async_commit();
  }
  for (int t = 0; t < n_tiles; ++t) {
    cp_async_wait<Cfg::STAGES - 2>();
    if (by_keys) __syncwarp(); else __syncthreads();
    // the slot of tile t - 1 takes tile t + STAGES - 1: every reader of it is past the barrier
    if (t + Cfg::STAGES - 1 < n_tiles) copy_tile(t + Cfg::STAGES - 1);
    cp_async_commit();
    const uint32_t st = ring + (t % Cfg::STAGES) * Cfg::STAGE;
    const int kb = k0 + t * kOwnTile;
    if (by_keys) {
      if (kb + warp * 16 < k1)
        score_group(st + warp * Cfg::GROUP, st + (kOwnWarps + warp) * Cfg::GROUP, kb + warp * 16);
    } else if (w_rho < end) {
#pragma unroll 1
      for (int w = 0; w < kOwnWarps; ++w)
        if (kb + w * 16 < k1) score_group(st + w * Cfg::GROUP, st + (kOwnWarps + w) * Cfg::GROUP, kb + w * 16);
    }
  }
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    l_lo += __shfl_xor_sync(0xffffffffu, l_lo, o);
    l_hi += __shfl_xor_sync(0xffffffffu, l_hi, o);
  }

  // ---- the unit's rows leave: as a part, or finished
  const int64_t slot = static_cast<int64_t>(part) * b.n_rows;
  auto place = [&](int rho) { return static_cast<int64_t>(row0 + rho / a.G) * a.Hq + g * a.G + rho % a.G; };
  auto put_ml = [&](int rho, float m, float l) {
    if (only) {
      if (a.lse) a.lse[place(rho)] = (m + log2f(l)) * 0.69314718055994531f;
    } else {
      parts.ml[slot * a.Hq + place(rho)] = make_float2(m, l);
    }
  };
  if (!by_keys) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int rho = half ? hi : lo;
      if (rho >= end) continue;
      const float m = half ? m_hi : m_lo, l = half ? l_hi : l_lo, inv = l > 0.f ? 1.f / l : 0.f;
      if ((lane & 3) == 0) put_ml(rho, m, l);
      if (only) {
        T* o = static_cast<T*>(a.o) + place(rho) * D;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          *reinterpret_cast<uint32_t*>(o + i * 8 + qc) = pack2<T>(acc[i][2 * half] * inv, acc[i][2 * half + 1] * inv);
      } else {
        float* o = parts.o + (slot * a.Hq + place(rho)) * D;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          *reinterpret_cast<float2*>(o + i * 8 + qc) = make_float2(acc[i][2 * half], acc[i][2 * half + 1]);
      }
    }
    return;
  }
  // the warps' sums of the same rows meet in the ring, now free
  cp_async_wait<0>();
  __syncthreads();
  float* so = reinterpret_cast<float*>(smem);
  float2* sml = reinterpret_cast<float2*>(smem + kOwnWarps * 16 * D * 4);
  {
    const int r = lane >> 2;
    if ((lane & 3) == 0) {
      sml[warp * 16 + r] = make_float2(m_lo, l_lo);
      sml[warp * 16 + r + 8] = make_float2(m_hi, l_hi);
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      *reinterpret_cast<float2*>(so + (warp * 16 + r) * D + i * 8 + qc) = make_float2(acc[i][0], acc[i][1]);
      *reinterpret_cast<float2*>(so + (warp * 16 + r + 8) * D + i * 8 + qc) = make_float2(acc[i][2], acc[i][3]);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * (D / 4); i += kOwnWarps * 32) {
    const int r = i / (D / 4), d = i % (D / 4) * 4;
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int w = 0; w < kOwnWarps; ++w) M = fmaxf(M, sml[w * 16 + r].x);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kOwnWarps; ++w) {
      const float2 ml = sml[w * 16 + r];
      const float f = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
      const float4 v = *reinterpret_cast<const float4*>(so + (w * 16 + r) * D + d);
      L += ml.y * f;
      s.x += v.x * f;
      s.y += v.y * f;
      s.z += v.z * f;
      s.w += v.w * f;
    }
    const int rho = rho0 + r;
    if (d == 0) put_ml(rho, M, L);
    if (only) {
      const float inv = L > 0.f ? 1.f / L : 0.f;
      *reinterpret_cast<uint2*>(static_cast<T*>(a.o) + place(rho) * D + d) =
          make_uint2(pack2<T>(s.x * inv, s.y * inv), pack2<T>(s.z * inv, s.w * inv));
    } else {
      *reinterpret_cast<float4*>(parts.o + (slot * a.Hq + place(rho)) * D + d) = s;
    }
  }
}

// ------------------------------------------------------------------ joining the parts
//
// One warp per (row, head): the parts' maxima and sums are read by lanes, then every lane adds
// its D / 32 output entries of each part.  Parts are added in a fixed order.
template <typename T, int D>
__global__ void __launch_bounds__(256) batch_combine_kernel(const PagedView c, const BatchView b, const AttnArgs a,
                                                            const SharedPlan p, const Parts parts) {
  constexpr int E = D >= 32 ? D / 32 : 1;
  const int w = static_cast<int>((static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5), lane = threadIdx.x & 31;
  const int row = w / a.Hq, h = w - row * a.Hq;
  if (row >= b.n_rows) return;
  const int seq = warp_seq_of_row(b, row);
  if (seq < 0) return;
  const SeqSpan s = seq_span(b, seq);
  if (row >= s.row0 + s.nq) return;
  const int n_own = (s.len + p.own_chunk - 1) / p.own_chunk;
  int n_pre = p.pre_parts;
  if (p.pre_tc) {   // the CTAs that share this row's unit
    const int unit = h / a.G * p.pre_row_blocks + row / p.pre_rows;
    n_pre = ((unit + 1) * p.pre_tiles - 1) / p.pre_share - unit * p.pre_tiles / p.pre_share + 1;
  }
  if (p.pre_parts == 0 && n_own == 1) return;   // already written
  const int n = n_pre + n_own;
  const int64_t stride = static_cast<int64_t>(b.n_rows) * a.Hq, at = static_cast<int64_t>(row) * a.Hq + h;
  auto slot = [&](int i) { return (i < n_pre ? i : p.pre_parts + i - n_pre) * stride + at; };
  float M = -INFINITY;
  for (int i = lane; i < n; i += 32) M = fmaxf(M, parts.ml[slot(i)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float L = 0.f;
  Vec<float, E> sum;
#pragma unroll
  for (int e = 0; e < E; ++e) sum.v[e] = 0.f;
  for (int i0 = 0; i0 < n; i0 += 32) {
    float f = 0.f;
    if (i0 + lane < n) {
      const float2 ml = parts.ml[slot(i0 + lane)];
      f = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
      L += ml.y * f;
    }
    const int m = min(32, n - i0);
#pragma unroll 4
    for (int i = 0; i < m; ++i) {
      const float fi = __shfl_sync(0xffffffffu, f, i);
      if (fi == 0.f || lane * E >= D) continue;   // a part without keys for this row holds no sums
      const Vec<float, E> v = *reinterpret_cast<const Vec<float, E>*>(parts.o + slot(i0 + i) * D + lane * E);
#pragma unroll
      for (int e = 0; e < E; ++e) sum.v[e] = fmaf(v.v[e], fi, sum.v[e]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  const float inv = L > 0.f ? 1.f / L : 0.f;
  if (lane * E < D) {
    Vec<T, E> r;
#pragma unroll
    for (int e = 0; e < E; ++e) r.v[e] = from_f32<T>(sum.v[e] * inv);
    *reinterpret_cast<Vec<T, E>*>(static_cast<T*>(a.o) + at * D + lane * E) = r;
  }
  if (a.lse && lane == 0) a.lse[at] = (M + log2f(L)) * 0.69314718055994531f;
}

// ------------------------------------------------------------------ host

static SharedPlan plan_shared(const PagedView& c, const BatchView& b, int Hq) {
  SharedPlan p = {};
  const int G = Hq / c.Hkv, sms = num_sms();
  auto chunks = [&](int64_t units, int len, int* chunk, int* n) {
    // parts of at least 128 keys, enough units to fill every SM four times, and none above 1024
    // keys, so that one long sequence does not outlast the others
    const int64_t fill = std::min<int64_t>((4 * sms + units - 1) / std::max<int64_t>(units, 1), (len + 127) / 128);
    const int want = static_cast<int>(std::max<int64_t>({1, fill, (len + 1023) / 1024}));
    *chunk = std::max(kOwnTile, ((len + want - 1) / want + kOwnTile - 1) / kOwnTile * kOwnTile);
    *n = (len + *chunk - 1) / *chunk;
  };
  p.own_row_blocks = std::max(1, (std::min(b.max_q, b.n_rows) * G + kOwnRows - 1) / kOwnRows);
  chunks(static_cast<int64_t>(b.n_seq) * c.Hkv * p.own_row_blocks, std::max(1, b.max_len), &p.own_chunk, &p.own_parts);
  // More than one 16-row MMA tile of score rows per KV head: tcgen05 (one tile has nothing to share,
  // and the warp-MMA kernel splits its keys over every SM).
  if (b.prefix_len > 0 && c.D >= 64 && b.n_rows * G > 16) {
    p.pre_tc = true;
    p.pre_rows = 2 * (128 / G);
    p.pre_row_blocks = (b.n_rows + p.pre_rows - 1) / p.pre_rows;
    p.pre_tiles = (b.prefix_len + 127) / 128;
    const int64_t total = static_cast<int64_t>(p.pre_row_blocks) * c.Hkv * p.pre_tiles;
    p.pre_share = static_cast<int>(std::max<int64_t>((total + sms - 1) / sms, std::min(2, p.pre_tiles)));
    p.pre_ctas = static_cast<int>((total + p.pre_share - 1) / p.pre_share);
    p.pre_parts = (p.pre_tiles + p.pre_share - 2) / p.pre_share + 1;   // CTAs that one unit can meet
  } else if (b.prefix_len > 0) {
    p.pre_row_blocks = (b.n_rows * G + kOwnRows - 1) / kOwnRows;
    chunks(static_cast<int64_t>(p.pre_row_blocks) * c.Hkv, b.prefix_len, &p.pre_chunk, &p.pre_parts);
  }
  return p;
}

size_t parts_bytes(const SharedPlan& p, const BatchView& b, int Hq, int D) {
  const int n = p.pre_parts + p.own_parts;
  if (n <= 1) return 0;
  const size_t rows = static_cast<size_t>(n) * b.n_rows * Hq;
  return align_up(rows * D * sizeof(float), 256) + align_up(rows * sizeof(float2), 256);
}

template <typename T, int D>
static qcf_status shared_prefix_attn_launch(const qcf_paged_kv* cache, const PagedView& c, const BatchView& b, const AttnArgs& a, const SharedPlan& p,
                                            Parts parts, cudaStream_t st) {
  const char* who = "qcf_shared_prefix_attn";
  using Cfg = OwnCfg<D>;
  static PerDevice<cudaError_t> smem_attr;
  const cudaError_t attr = smem_attr.get(current_device(), [] {
    return cudaFuncSetAttribute(own_attn_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM);
  });
  if (attr != cudaSuccess) return cuda_error(attr, "qcf_shared_prefix_attn: smem attribute");
  const int64_t pre_units = p.pre_tc ? 0 : static_cast<int64_t>(p.pre_parts) * p.pre_row_blocks * c.Hkv;
  const int64_t units = pre_units + static_cast<int64_t>(b.n_seq) * p.own_row_blocks * p.own_parts * c.Hkv;
  if (units > INT32_MAX) return set_error(QCF_ERR_SHAPE, "%s: %lld units of work are too many for one call", who, (long long)units);
  if (p.pre_tc) {
    const qcf_status s = prefix_tc_launch(cache, c, b, a, p, parts, st);
    if (s != QCF_OK) return s;
  }
  {
    LaunchScope ls(KC_OWN_ATTN, st);
    own_attn_kernel<T, D><<<static_cast<unsigned>(units), kOwnWarps * 32, Cfg::SMEM, st>>>(
        c, b, a, p, parts, static_cast<int>(pre_units), device_status_ptr());
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_error(e, "qcf_shared_prefix_attn: launch");
  }
  if (p.pre_parts + p.own_parts > 1) {
    LaunchScope ls(KC_BATCH_COMBINE, st);
    const int64_t warps = static_cast<int64_t>(b.n_rows) * a.Hq;
    batch_combine_kernel<T, D><<<static_cast<unsigned>((warps + 7) / 8), 256, 0, st>>>(c, b, a, p, parts);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_error(e, "qcf_shared_prefix_attn: combine launch");
  }
  return QCF_OK;
}

template <typename T>
static qcf_status shared_prefix_attn_type(const qcf_paged_kv* cache, const PagedView& c, const BatchView& b, const AttnArgs& a, const SharedPlan& p,
                                          Parts parts, cudaStream_t st) {
  switch (c.D) {
    case 16: return shared_prefix_attn_launch<T, 16>(cache, c, b, a, p, parts, st);
    case 64: return shared_prefix_attn_launch<T, 64>(cache, c, b, a, p, parts, st);
    default: return shared_prefix_attn_launch<T, 128>(cache, c, b, a, p, parts, st);
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
  if (b.n_seq == 0 || b.n_rows == 0) return 0;
  return parts_bytes(plan_shared(c, b, Hq), b, Hq, c.D);
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
  if (take_fault(2)) return set_error(QCF_ERR_WORKSPACE, "%s: injected short workspace", who);
  if (b.n_seq == 0 || b.n_rows == 0) return QCF_OK;
  const SharedPlan p = plan_shared(c, b, Hq);
  const size_t need = parts_bytes(p, b, Hq, c.D);
  if (need && (!ws || ws_bytes < need)) return set_error(QCF_ERR_WORKSPACE, "%s: workspace %zu < %zu", who, ws_bytes, need);
  const size_t rows = static_cast<size_t>(p.pre_parts + p.own_parts) * b.n_rows * Hq;
  const Parts parts{static_cast<float*>(ws),
                    reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + align_up(rows * c.D * sizeof(float), 256))};
  const AttnArgs a{q, q_stride, cache->k, cache->v, o, lse, Hq, Hq / c.Hkv, scale * 1.4426950408889634f};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return cache->dtype == QCF_BF16 ? shared_prefix_attn_type<__nv_bfloat16>(cache, c, b, a, p, parts, st)
                                  : shared_prefix_attn_type<__half>(cache, c, b, a, p, parts, st);
}

}  // extern "C"
