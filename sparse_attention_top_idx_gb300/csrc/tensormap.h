// tensormap.h -- the CUDA driver API's tensor-map encoder (defined in api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

namespace dsaidx {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled, looked up at run time; null when missing.
EncodeTiledFn encode_tiled_fn();

// The encoder wants a current context, which a thread has only after its first
// runtime call that needs one.  A call that fails binds the current device's
// context to the thread and is made once more.
template <class... Args>
inline CUresult encode_tiled(EncodeTiledFn enc, Args... args) {
    CUresult r = enc(args...);
    int dev = 0;
    if (r != CUDA_SUCCESS && cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess) r = enc(args...);
    return r;
}

}  // namespace dsaidx
