// What the kernels of the shared-prefix attention share: arguments, the split of the work into
// parts, and where each part leaves its sums.
#pragma once

#include "paged.cuh"

namespace qcf {

struct AttnArgs {
  const void* q;
  int64_t q_stride;
  void* o;
  float* lse;
  int Hq, G;          // G = Hq / Hkv
  uint32_t g_mul;     // ceil(2^32 / G): n / G as a product, for n < 2^28 (an integer division takes a warp over 100 cycles)
  float scale_log2;   // scale * log2(e): logits are kept in powers of two
};

// Weights are powers 2^(x - m).  m follows the maximum of the logits x by steps of more than 2^8, so
// they stay below 2^8 above their first maximum; in fp16 m lies 7 below that maximum, so that weights
// down to 2^-21 of the largest are normal numbers (the top ones below 2^15), and many small
// weights next to a large one keep their bits.  bf16 has the exponents of fp32.
template <typename T>
constexpr float kWeightLift = std::is_same<T, __half>::value ? 7.f : 0.f;

__device__ __forceinline__ int div_g(const AttnArgs& a, int n) {
  return a.G == 1 ? n : static_cast<int>(__umulhi(static_cast<uint32_t>(n), a.g_mul));
}

// Every part (a range of keys of the prefix, or of a sequence's own tokens) of a row and head
// leaves its unnormalised output (fp32 [D]), maximum and sum of powers of two; the combine kernel
// joins them.  A row whose only part is the whole of its sequence is written to o at once.
//
// The prefix on tcgen05 (pre_tc): either every (row block, KV head) unit in pre_parts equal parts, a
// CTA each (pre_even), or the key tiles of all units dealt out evenly, pre_share to a CTA, a part
// being the CTA's place among those that share the unit.
// The stream (own tokens, and the prefix where tcgen05 does not take it): the 32-key tiles of all
// (sequence, block of 16 score rows, KV head) units, dealt out in the same way over `workers`
// warps, by lengths that are read on the device.  Part 0 of a unit has a slot per row; a later part
// begins where a worker's share begins, so each worker has one slot for it.
struct SharedPlan {
  bool pre_tc, pre_even;
  int pre_row_blocks, pre_rows, pre_tiles, pre_share, pre_ctas, pre_parts;
  bool pre_stream;                   // the prefix is part of the stream
  int stream_blocks, stream_tiles;   // its blocks of 16 score rows and key tiles
  int ctas, workers;
};
constexpr int kStreamRows = 16;      // score rows of a stream unit
constexpr int kStreamKeys = 32;      // keys of a tile
constexpr int kMinShare = 2;         // tiles dealt to a worker at least

struct Workspace {
  float* tc_o;        // [pre_parts][n_rows][Hq][D]
  float2* tc_ml;      // [pre_parts][n_rows][Hq]: maximum, sum
  float* own_o;       // [n_rows][Hq][D]: part 0 of the own tokens
  float2* own_ml;
  float* pre_o;       // part 0 of a streamed prefix
  float2* pre_ml;
  float* spill_o;     // [workers][16][D]: the part a worker's share begins in the middle of
  float2* spill_ml;
  int4* rows;         // [n_rows]: row of its sequence (-1: of none), the sequence's first tile, tiles of its length
  int* share;         // tiles dealt to a worker
};
size_t workspace_layout(const SharedPlan& p, const BatchView& b, int Hq, int D, void* base, Workspace* w);

// The tensor-core kernel of the prefix (prefix_attn.cu): its parts of every row of the batch.
qcf_status prefix_tc_launch(const qcf_paged_kv* cache, const PagedView& c, const BatchView& b, const AttnArgs& a,
                            const SharedPlan& p, const Workspace& w, cudaStream_t st);

__device__ __forceinline__ void tma_load_4d(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];"
      ::"r"(smem_u32(smem_dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

// Tensor map of the pages: entries of a head, rows of a page, heads, pages; boxes of `rows` rows
// and `cols` entries of one head and page.
inline bool encode_pages(CUtensorMap* map, const void* base, const PagedView& c, int rows, int cols, CUtensorMapSwizzle sw) {
  const uint64_t dims[4] = {static_cast<uint64_t>(c.D), static_cast<uint64_t>(1) << c.page_shift, static_cast<uint64_t>(c.Hkv),
                            static_cast<uint64_t>(c.n_pages)};
  const uint64_t strides[3] = {static_cast<uint64_t>(c.row_stride) * 2, static_cast<uint64_t>(c.head_stride) * 2,
                               static_cast<uint64_t>(c.page_stride) * 2};
  const uint32_t box[4] = {static_cast<uint32_t>(cols), static_cast<uint32_t>(rows), 1, 1};
  return encode_tmap_4d(map, base, dims, strides, box, sw);
}

// m16n8k16 on warp tensor cores, both 16-bit types, fp32 sums.
template <typename T>
__device__ __forceinline__ void mma_16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma_16816<__nv_bfloat16>(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  mma_bf16_16816(c, a, b0, b1);
}
template <>
__device__ __forceinline__ void mma_16816<__half>(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  return pack_bf16x2(lo, hi);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Named barrier over the `count` threads that meet at `id`.
__device__ __forceinline__ void bar_sync(int id, int count) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
}

// 32 lanes x 128 consecutive 32-bit columns in one load; the wait sits in the same statement so no
// register is read before the data has landed.
__device__ __forceinline__ void tmem_ld128(uint32_t taddr, float* v) {
  uint32_t r[128];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x128.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
      "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63, "
      "%64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, %77, %78, %79, "
      "%80, %81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, %95, "
      "%96, %97, %98, %99, %100, %101, %102, %103, %104, %105, %106, %107, %108, %109, %110, %111, "
      "%112, %113, %114, %115, %116, %117, %118, %119, %120, %121, %122, %123, %124, %125, %126, %127}, [%128];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
        "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63]),
        "=r"(r[64]), "=r"(r[65]), "=r"(r[66]), "=r"(r[67]), "=r"(r[68]), "=r"(r[69]), "=r"(r[70]), "=r"(r[71]),
        "=r"(r[72]), "=r"(r[73]), "=r"(r[74]), "=r"(r[75]), "=r"(r[76]), "=r"(r[77]), "=r"(r[78]), "=r"(r[79]),
        "=r"(r[80]), "=r"(r[81]), "=r"(r[82]), "=r"(r[83]), "=r"(r[84]), "=r"(r[85]), "=r"(r[86]), "=r"(r[87]),
        "=r"(r[88]), "=r"(r[89]), "=r"(r[90]), "=r"(r[91]), "=r"(r[92]), "=r"(r[93]), "=r"(r[94]), "=r"(r[95]),
        "=r"(r[96]), "=r"(r[97]), "=r"(r[98]), "=r"(r[99]), "=r"(r[100]), "=r"(r[101]), "=r"(r[102]), "=r"(r[103]),
        "=r"(r[104]), "=r"(r[105]), "=r"(r[106]), "=r"(r[107]), "=r"(r[108]), "=r"(r[109]), "=r"(r[110]), "=r"(r[111]),
        "=r"(r[112]), "=r"(r[113]), "=r"(r[114]), "=r"(r[115]), "=r"(r[116]), "=r"(r[117]), "=r"(r[118]), "=r"(r[119]),
        "=r"(r[120]), "=r"(r[121]), "=r"(r[122]), "=r"(r[123]), "=r"(r[124]), "=r"(r[125]), "=r"(r[126]), "=r"(r[127])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 128; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Two fp32 values in one register pair, for the instructions that work on both.
struct Pair {
  uint64_t v;
};
__device__ __forceinline__ Pair make_pair2(float lo, float hi) {
  Pair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p.v) : "f"(lo), "f"(hi));
  return p;
}
__device__ __forceinline__ void split(Pair p, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p.v));
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return d;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}

}  // namespace qcf
