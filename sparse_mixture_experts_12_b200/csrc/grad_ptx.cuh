// tcgen05 / TMA building blocks of the gradients' kernels beside those of tc_ptx.cuh.
#pragma once

#include "tc_ptx.cuh"

namespace moe {
namespace tc {

// Shared-memory descriptor (see sw128_desc) of an operand whose M (or N) index is the
// contiguous one: 64-element blocks of it, each K rows of 128 bytes (8-row swizzle atoms,
// 1024 bytes apart along K), follow each other every `block_bytes`. A K = 16 step is 2048
// bytes.
__device__ __forceinline__ uint64_t sw128_desc_mn(uint32_t saddr, uint32_t block_bytes) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)(block_bytes >> 4) << 16;   // leading-dim byte offset: the next block
  d |= (uint64_t)(1024 >> 4) << 32;          // stride-dim byte offset: the next 8 K rows
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
constexpr uint32_t kIdescMnA = 1u << 15, kIdescMnB = 1u << 16;  // A, B not K-major

// mbar_arrive_cluster where no memory writes are handed over with it (tensor memory that
// has been read): without the release at cluster scope, which waits for the thread's
// stores, some 2000 clocks.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// (see tma_load_2d_pair)
__device__ __forceinline__ void tma_load_3d_pair(const CUtensorMap *map, uint32_t mbar_cluster,
                                                 void *dst, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(mbar_cluster), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// ------------------------------------------------------------------ host side
// make_map with rows `ld` elements apart.
inline bool make_map_ld(CUtensorMap *map, const void *ptr, uint64_t rows, uint64_t cols,
                        uint32_t box_rows, uint64_t ld) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {ld * 2};
  cuuint32_t box[2] = {(cuuint32_t)kBlockK, box_rows};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(ptr), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// The bf16 matrix (rows `ld` elements apart, 0: cols) as [cols / 64, rows, 64]: a box of two
// 64-column blocks of 64 rows lands block after block (the layout of sw128_desc_mn). cols: a
// multiple of 64.
inline bool make_mn_map(CUtensorMap *map, const void *ptr, uint64_t rows, uint64_t cols,
                        uint64_t ld = 0) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[3] = {(cuuint64_t)kBlockK, rows, cols / kBlockK};
  cuuint64_t strides[2] = {(ld ? ld : cols) * 2, kBlockK * 2};
  cuuint32_t box[3] = {(cuuint32_t)kBlockK, (cuuint32_t)kBlockK, 2};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// 2-D fp32 map for TMA stores of 32 x 32 tiles (128-byte rows, 128-byte swizzle).
inline bool make_f32_map(CUtensorMap *map, void *ptr, uint64_t rows, uint64_t cols) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols * 4};
  cuuint32_t box[2] = {(cuuint32_t)kStoreBox, (cuuint32_t)kStoreBox};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, ptr, dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

}  // namespace tc
}  // namespace moe
