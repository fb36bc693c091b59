// Boxes of 8-bit pages: the 16 slots of a step, for one head, in one TMA copy.
//
// The pages' codes are a tensor (values, slots of a page, heads, pages) with the pages' own strides.  A step of 16 slots is
// aligned to 16, and page_size is a multiple of 16, so a step is a box inside one page.
#pragma once

#include <cuda.h>

#include "cache_device.cuh"
#include "specdec_device.cuh"

namespace specdec {

constexpr int kBoxSlots = 16;

struct Maps {
  CUtensorMap k, v;
  int heads, pages;  // 0: all heads, or pages, lie at the same place (a stride of 0): the coordinate is 0
};

// One box of keys (or values) to shared memory: rows of head_dim bytes.
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap* map, int slot, int head, int page, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(0), "r"(slot), "r"(head), "r"(page), "r"(smem_addr(bar))
      : "memory");
}

// (By the runtime's lookup of the driver's function: the library needs no link to the driver's.)
inline cudaError_t encode_maps(const Pages& pg, bool swizzled_k, bool swizzled_v, Maps* maps) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess || q != cudaDriverEntryPointSuccess)
      return static_cast<Encode>(nullptr);
    return reinterpret_cast<Encode>(f);
  }();
  if (!encode) return cudaErrorNotSupported;
  maps->heads = pg.head_stride != 0;
  maps->pages = pg.page_stride != 0;
  const cuuint64_t D = static_cast<cuuint64_t>(pg.head_dim);
  const cuuint64_t dims[4] = {D, static_cast<cuuint64_t>(pg.page_size), maps->heads ? static_cast<cuuint64_t>(pg.kv_heads) : 1,
                              maps->pages ? static_cast<cuuint64_t>(pg.num_pages) : 1};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(pg.slot_stride), static_cast<cuuint64_t>(maps->heads ? pg.head_stride : pg.slot_stride),
                                 static_cast<cuuint64_t>(maps->pages ? pg.page_stride : pg.slot_stride)};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(D), kBoxSlots, 1, 1}, one[4] = {1, 1, 1, 1};
  const CUtensorMapSwizzle rows = D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  for (int i = 0; i < 2; ++i)
    if (encode(i ? &maps->v : &maps->k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, i ? pg.v : pg.k, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               (i ? swizzled_v : swizzled_k) ? rows : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  return cudaSuccess;
}

// What a warp knows of 32 steps of its own, a lane each: the page, its slot, and the scale bytes of the block.
struct Look {
  int page, in_page;          // page -1: no such step; num_pages: out of range
  uint32_t scale_k, scale_v;  // (nothing is made of the bytes before they are used: it would wait for them)
  __device__ __forceinline__ void find(const Pages& pg, const int32_t* table, int slot, bool there) {
    page = -1;
    in_page = 0;
    scale_k = scale_v = 0;
    if (!there) return;
    const int logical = page_of(pg, slot), p = __ldg(table + logical);
    page = static_cast<unsigned>(p) < static_cast<unsigned>(pg.num_pages) ? p : pg.num_pages;
    in_page = slot - logical * pg.page_size;
  }
  __device__ __forceinline__ void find_scales(const Pages& pg, int head) {
    if (static_cast<unsigned>(page) >= static_cast<unsigned>(pg.num_pages)) return;
    const int64_t so = page * pg.scale_page_stride + block_of(pg, in_page) * pg.scale_slot_stride + head * pg.scale_head_stride;
    scale_k = __ldg(reinterpret_cast<const uint8_t*>(pg.k_scales) + so);
    scale_v = __ldg(reinterpret_cast<const uint8_t*>(pg.v_scales) + so);
  }
};

}  // namespace specdec
