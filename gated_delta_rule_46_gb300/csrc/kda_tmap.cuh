// kda_tmap.cuh -- host side: TMA descriptors of row-major tensors.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace kda {

typedef CUresult (*TmapEncode)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                               const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                               CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline TmapEncode tmap_encode() {
    static const TmapEncode enc = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) !=
                cudaSuccess || q != cudaDriverEntryPointSuccess)
            ptr = nullptr;
        return reinterpret_cast<TmapEncode>(ptr);
    }();
    return enc;
}

// A [rows][cols] tensor of 2- (bf16) or 4-byte (float32) elements, rows
// row_bytes apart (a multiple of 16, as is the base address), in boxes of
// box_rows x 128 bytes with the 128-byte swizzle; reads outside give zeros.
inline bool make_map_2d(CUtensorMap *m, const void *base, bool bf16, uint64_t rows, uint64_t cols, uint64_t row_bytes,
                        uint32_t box_rows) {
    const TmapEncode enc = tmap_encode();
    if (!enc) return false;
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {row_bytes};
    const cuuint32_t box[2] = {bf16 ? 64u : 32u, box_rows}, one[2] = {1, 1};
    return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
               const_cast<void *>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A dense [pages][heads][rows][D] tensor of bytes, D = 32, 64 or 128, in boxes of whole rows with the swizzle of their
// size.  (An axis each: rows of all pages counted in one would pass the 31 bits of a coordinate.)
inline bool make_map_pages(CUtensorMap *m, const void *base, uint64_t pages, uint64_t heads, uint64_t rows, int D,
                           uint32_t box_rows) {
    const TmapEncode enc = tmap_encode();
    if (!enc) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)D, rows, heads, pages};
    const cuuint64_t strides[3] = {(cuuint64_t)D, D * rows, D * rows * heads};
    const cuuint32_t box[4] = {(cuuint32_t)D, box_rows, 1, 1}, one[4] = {1, 1, 1, 1};
    const CUtensorMapSwizzle sw = D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                  : D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B;
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(base), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A bf16 [tokens][heads][d] tensor, tokens row_bytes apart (a multiple of 16), in boxes of one head's 64 channels x
// box_tokens; channels outside read as zeros and are not written.
inline bool make_map_heads(CUtensorMap *m, const void *base, uint64_t tokens, uint64_t heads, uint64_t d, uint64_t row_bytes,
                           uint32_t box_tokens) {
    const TmapEncode enc = tmap_encode();
    if (!enc) return false;
    const cuuint64_t dims[3] = {d, heads, tokens}, strides[2] = {d * 2, row_bytes};
    const cuuint32_t box[3] = {64u, 1u, box_tokens}, one[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace kda
