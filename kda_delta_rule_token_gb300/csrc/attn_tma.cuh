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
inline PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
        return nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
}

inline bool make_cache_map(CUtensorMap* m, const AttnLayer& l, const void* cache, int box_rows, int blocks) {
    const auto fn = map_encoder();
    if (!fn) return false;
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

// The bf16 cache as (64 channels, row of eight, half of the channels, eight of
// the page's rows, page and head), boxes of box_rows whole rows: in shared
// memory each eight rows are two swizzled 1024-byte atoms, lower and upper
// channels, and eights follow each other evenly across pages of any size, as a
// tensor-core operand wants them (either way round), with one copy per page.
inline bool make_cache_map_atoms(CUtensorMap* m, const AttnLayer& l, const void* cache, int box_rows) {
    const auto fn = map_encoder();
    if (!fn) return false;
    const cuuint64_t dims[5] = {64, 8, 2, (cuuint64_t)l.page_size / 8, (cuuint64_t)l.num_pages * l.Hkv};
    const cuuint64_t strides[4] = {256, 128, 2048, (cuuint64_t)l.page_size * 256};
    const cuuint32_t box[5] = {64, 8, 2, (cuuint32_t)box_rows / 8, 1};
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(cache), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace kda
