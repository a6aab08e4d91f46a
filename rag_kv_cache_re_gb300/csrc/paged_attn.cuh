// What the kernels of the shared-prefix attention share: arguments, the split of the work into
// parts, and where each part leaves its sums.
#pragma once

#include "paged.cuh"

namespace qcf {

struct AttnArgs {
  const void* q;
  int64_t q_stride;
  const void* k;
  const void* v;
  void* o;
  float* lse;
  int Hq, G;          // G = Hq / Hkv
  float scale_log2;   // scale * log2(e): logits are kept in powers of two
};

// Every part (a range of keys of the prefix, or of a sequence's own tokens) of a row and head
// leaves its unnormalised output, maximum and sum of powers of two; the combine kernel joins
// them.  A row whose only part is its sequence's single own one is written at once.
//   o   [part][n_rows][Hq][D] fp32      ml  [part][n_rows][Hq] (maximum, sum)
struct Parts {
  float* o;
  float2* ml;
};

struct SharedPlan {
  // own tokens: chunks of own_chunk keys (a multiple of the tile), at most own_parts of them
  int own_chunk, own_parts, own_row_blocks;
  // prefix: pre_parts slots per row.  On the warp-MMA kernel a part is a chunk of pre_chunk keys;
  // on the tensor-core kernel the tiles of all (row block, KV head) units are dealt out evenly,
  // pre_share to a CTA, and the part is the CTA's place among those that share the unit.
  int pre_parts, pre_chunk, pre_row_blocks;
  bool pre_tc;
  int pre_rows, pre_tiles, pre_share, pre_ctas;   // tensor-core kernel: rows of q per unit, key tiles
};

size_t parts_bytes(const SharedPlan& p, const BatchView& b, int Hq, int D);

// The tensor-core kernel of the prefix (prefix_attn.cu): its parts of every row of the batch.
qcf_status prefix_tc_launch(const qcf_paged_kv* cache, const PagedView& c, const BatchView& b, const AttnArgs& a,
                            const SharedPlan& p, Parts parts, cudaStream_t st);

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

__device__ __forceinline__ void cp_async16(uint32_t smem, const void* src, bool take) {   // zeros when not taken
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(src), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace qcf
