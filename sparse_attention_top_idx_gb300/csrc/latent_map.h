// latent_map.h -- the tensor map of a [rows, heads, dim] bf16 tensor with any
// positive strides, 128-byte swizzled boxes of 64 values.
#pragma once

#include <stdint.h>

#include <utility>

#include "tensormap.h"

namespace dsaidx {

// Boxes of box_heads x box_rows (one of them 1), 64 values each.  The map's
// middle dimension is the one with the smaller stride: *swap is set when that
// is the row, and coordinates are then (value, row, head).  Values outside
// the tensor read as zeros.
inline bool head_map(CUtensorMap* map, EncodeTiledFn enc, const void* base, int dim, int64_t row_stride,
                     int64_t head_stride, int64_t rows, int heads, int box_heads, int box_rows, int* swap) {
    if (heads == 1) head_stride = dim;             // strides nobody steps over
    if (rows == 1) row_stride = head_stride * heads;
    *swap = head_stride > row_stride;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_stride) * 2, static_cast<cuuint64_t>(row_stride) * 2};
    cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_rows)}, one[3] = {1, 1, 1};
    if (*swap) {
        std::swap(dims[1], dims[2]);
        std::swap(strides[0], strides[1]);
        std::swap(box[1], box[2]);
    }
    return encode_tiled(enc, map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, one,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace dsaidx
