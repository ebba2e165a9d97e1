// tensor_map.cuh -- tensor maps of caches, for copies by TMA.
#pragma once

#include <cuda.h>

#include "paged_attention.cuh"

namespace bevpool {

namespace {

// The driver's tensor-map encoder, found through the runtime.
using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                 const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

// A cache of codes as a tensor (element, slot, head, page) in boxes of `rows` slots
// (a page's, if it has fewer); swizzled: by the width of a row, 128 or 64 bytes.
inline bool code_map(const AttnArgs &a, const void *cache, int rows, bool swizzled, CUtensorMap *map) {
    const EncodeTiled encode = encode_tiled();
    if (!encode) return false;
    // the stride of an axis of one entry is never used
    const auto stride = [&](int64_t s, int64_t n) { return static_cast<cuuint64_t>(n > 1 ? s : a.D); };
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(a.D), static_cast<cuuint64_t>(a.pg.page_size), static_cast<cuuint64_t>(a.Hk),
                                static_cast<cuuint64_t>(a.pg.n_pages)};
    const cuuint64_t strides[3] = {stride(a.pg.slot_stride, a.pg.page_size), stride(a.pg.head_stride, a.Hk),
                                   stride(a.pg.page_stride, a.pg.n_pages)};
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(a.D), static_cast<cuuint32_t>(a.pg.page_size < rows ? a.pg.page_size : rows), 1, 1};
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(cache), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  !swizzled ? CU_TENSOR_MAP_SWIZZLE_NONE : a.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

}  // namespace bevpool
