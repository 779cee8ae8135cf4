// Tensor maps of token rows, [T, D] elements a stride apart, for TMA loads and stores of boxes of them.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/kda.h"

namespace kda {
namespace layer {

// [T, D] rows a stride apart in boxes of `rows` rows and `width` channels.  Needs 16-byte aligned rows.
inline bool make_row_map(CUtensorMap *m, const void *base, int64_t T, int D, int64_t stride, kda_dtype_t dtype, int width, int rows) {
    typedef CUresult (*encode_fn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                  const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                  CUtensorMapFloatOOBfill);
    static const encode_fn encode = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return (encode_fn)p;
    }();
    if (!encode) return false;
    const int64_t es = dtype == KDA_BF16 ? 2 : 4;
    const cuuint64_t dims[3] = {(cuuint64_t)D, 1, (cuuint64_t)T};
    const cuuint64_t strides[2] = {(cuuint64_t)(stride * es), (cuuint64_t)(stride * es)};
    const cuuint32_t box[3] = {(cuuint32_t)width, 1, (cuuint32_t)rows}, estr[3] = {1, 1, 1};
    return encode(m, dtype == KDA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void *>(base), dims,
                  strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace layer
}  // namespace kda
