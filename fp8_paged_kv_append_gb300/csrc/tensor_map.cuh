// Host side: the TMA tensor maps of query / output rows and of the key pool.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "k16v8_device.cuh"

namespace k16v8 {

static inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    cudaDriverEntryPointQueryResult q;
    void *p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  return fn;
}

// fp16 [tokens][heads][128] in boxes of 64 dims x 4 heads x 32 tokens (half a
// 128-row operand tile), 128-byte swizzle.
static inline bool map_rows(CUtensorMap *m, const void *rows, int32_t heads, int32_t tokens) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(kHeadDim), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(tokens)};
  const cuuint64_t strides[2] = {kHeadDim * 2ull, static_cast<cuuint64_t>(heads) * kHeadDim * 2ull};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(kGroup), 32};
  const cuuint32_t es[3] = {1, 1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(rows), dims, strides, box,
                es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The key pool as fp16 [rows][128] in boxes of 64 dims x one page, 128-byte
// swizzle.
static inline bool map_keys(CUtensorMap *m, const void *k_cache, uint64_t rows) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(kHeadDim), rows};
  const cuuint64_t strides[1] = {kHeadDim * 2ull};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(kPage)};
  const cuuint32_t es[2] = {1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void *>(k_cache), dims, strides,
                box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace k16v8
