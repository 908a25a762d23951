// tensormap.h -- the CUDA driver API's tensor-map encoder (defined in api.cu).
#pragma once

#include <cuda.h>

namespace dsaidx {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled, looked up at run time; null when missing.
EncodeTiledFn encode_tiled_fn();

}  // namespace dsaidx
