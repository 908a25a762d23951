// qlatent.h -- host structures and the block layout of the 8-bit latent cache,
// shared by its C ABI layer (qlatent_api.cu) and its kernels.  Not part of the
// public interface.
#pragma once

#include "dsaidx_qlatent.h"
#include "latent.h"

namespace dsaidx {

constexpr int kQRow = IDX_QLATENT_ROW_BYTES;
constexpr int kQCodes = IDX_LATENT_DIM;              // bytes of a row in front of the position part

// [block_size rows][block_size scales], rounded up to 128 bytes.
__host__ __device__ inline int64_t qlatent_block_bytes(int block_size) {
    return (static_cast<int64_t>(block_size) * (kQRow + 4) + 127) / 128 * 128;
}

struct QAppendArgs {
    AppendArgs a;
    int block_size;
    int64_t block_bytes;
};
cudaError_t launch_qappend(const QAppendArgs& a, cudaStream_t st);

struct QReadArgs {
    const void* pool;
    const int64_t* slots;
    void* out;
    int64_t n, out_stride, num_slots, block_bytes;
    int block_size;
    int32_t* status;
};
cudaError_t launch_qread(const QReadArgs& a, cudaStream_t st);

cudaError_t launch_qattend(const AttendArgs& a, int64_t block_bytes, cudaStream_t st);
size_t qattend_ws_need(int64_t rows, int heads, int64_t max_keys, bool paged);   // never above attend_ws_bytes

}  // namespace dsaidx
