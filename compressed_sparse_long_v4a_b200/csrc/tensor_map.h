// tensor_map.h -- tensor maps of the serving kernels' bf16 operands (host).
#pragma once

#include <cudaTypedefs.h>

#include "internal.h"

namespace v4a {

// [n][rows][d] bf16 viewed as (64 columns, rows, d / 64 slabs, n): a box is box_rows rows of `slabs` slabs and lands as slabs
// of box_rows rows of 128 bytes, swizzled.  False where the driver does not take it.
inline bool make_slab_map(CUtensorMap* map, const void* base, long long n, long long rows, int d, int box_rows, int slabs) {
    static const auto encode = []() -> PFN_cuTensorMapEncodeTiled_v12000 {  // once, whichever host thread comes first
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        return cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess && q == cudaDriverEntryPointSuccess
                   ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p)
                   : nullptr;
    }();
    if (!encode) return false;
    cuuint64_t dims[4] = {64, (cuuint64_t)rows, (cuuint64_t)(d / 64), (cuuint64_t)n};
    cuuint64_t strides[3] = {(cuuint64_t)d * 2, 128, (cuuint64_t)rows * d * 2};
    cuuint32_t box[4] = {64, (cuuint32_t)box_rows, (cuuint32_t)slabs, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline size_t align256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace v4a
