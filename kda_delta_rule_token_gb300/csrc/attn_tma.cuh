// Tensor maps of a bound key/value cache.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "attn_internal.cuh"

namespace kda {

// The cache [rows = pages * heads][page_size][128] as (128-byte column block,
// row in page, column block, page and head): boxes of one column block or of
// all (`blocks`), box_rows rows, 128-byte swizzle.  The column blocks (two in
// bf16, one in e4m3) come after the rows, so that a box lies in shared memory
// block by block, each of box_rows rows of 128 bytes.  Boxes outside the
// tensor read as zeros.
inline bool make_cache_map(CUtensorMap* m, const AttnLayer& l, const void* cache, int box_rows, int blocks) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
        return false;
    const auto fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    const int es = l.e4m3 ? 1 : 2;
    const cuuint64_t dims[4] = {(cuuint64_t)(128 / es), (cuuint64_t)l.page_size, (cuuint64_t)es,
                                (cuuint64_t)l.num_pages * l.Hkv};
    const cuuint64_t strides[3] = {(cuuint64_t)kHeadDim * es, 128, (cuuint64_t)l.page_size * kHeadDim * es};
    const cuuint32_t box[4] = {(cuuint32_t)(128 / es), (cuuint32_t)box_rows, (cuuint32_t)blocks, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(m, l.e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
              const_cast<void*>(cache), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace kda
