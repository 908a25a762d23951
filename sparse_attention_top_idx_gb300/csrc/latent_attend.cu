// latent_attend.cu -- absorbed latent attention over selected slots or a paged
// context: one CTA a (row, head), keys in tiles of 128, one pass with the
// running maximum and sum of the softmax in fp32.
#include <cuda_bf16.h>

#include <cmath>

#include "common.cuh"
#include "latent.h"

namespace dsaidx {

namespace {

constexpr int kTile = 128;

__device__ __forceinline__ float bf(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

// Slot of key j of a row, -1 where it is masked.
__device__ __forceinline__ int64_t key_slot(const AttendArgs& a, int64_t row, int j) {
    int64_t s;
    if (a.block_table == nullptr) {
        s = a.slots[row * a.slots_stride + j];
        if (s < 0) return -1;
    } else {
        const int blk = a.block_table[row * a.mbps + j / a.block_size];
        s = blk < 0 ? a.num_slots : static_cast<int64_t>(blk) * a.block_size + j % a.block_size;
    }
    if (s >= a.num_slots) {
        set_status(a.status, IDX_ERR_DEVICE_CHECK);
        return -1;
    }
    return s;
}

__global__ void __launch_bounds__(kTile) attend_kernel(const AttendArgs a) {
    __shared__ float q[IDX_LATENT_RECORD];
    __shared__ float pr[kTile];
    __shared__ int64_t sl[kTile];
    __shared__ float red[4];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t row = blockIdx.x;
    const int h = blockIdx.y, tid = threadIdx.x;
    const uint16_t* pool = static_cast<const uint16_t*>(a.pool);
    for (int i = tid; i < IDX_LATENT_RECORD; i += kTile)
        q[i] = i < IDX_LATENT_DIM ? bf(static_cast<const uint16_t*>(a.ql)[row * a.ql_row + h * a.ql_head + i])
                                  : bf(static_cast<const uint16_t*>(a.qp)[row * a.qp_row + h * a.qp_head + i - IDX_LATENT_DIM]);
    int n = a.max_keys;
    if (a.block_table != nullptr) {
        n = a.seq_lens[row];
        if (n < 0 || n > a.max_keys || n > static_cast<int64_t>(a.mbps) * a.block_size) {
            set_status(a.status, IDX_ERR_DEVICE_CHECK);
            n = 0;
        }
    }
    float m = -INFINITY, l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int j0 = 0; j0 < n; j0 += kTile) {
        __syncthreads();
        const int64_t slot = j0 + tid < n ? key_slot(a, row, j0 + tid) : -1;
        sl[tid] = slot;
        float s = -INFINITY;
        if (slot >= 0) {
            const uint16_t* r = pool + slot * IDX_LATENT_RECORD;
            s = 0.0f;
            for (int i = 0; i < IDX_LATENT_RECORD; ++i) s = fmaf(q[i], bf(r[i]), s);
            s *= a.scale;
        }
        float w = s;
        for (int k = 16; k > 0; k >>= 1) w = fmaxf(w, __shfl_xor_sync(~0u, w, k));
        if ((tid & 31) == 0) red[tid >> 5] = w;
        __syncthreads();
        const float mn = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
        if (mn == -INFINITY) continue;
        const float c = expf(m - mn);
        m = mn;
        pr[tid] = slot >= 0 ? expf(s - mn) : 0.0f;
        __syncthreads();
        l *= c;
        for (int i = 0; i < 4; ++i) o[i] *= c;
        for (int k = 0; k < kTile; ++k) {
            l += pr[k];
            if (sl[k] < 0) continue;
            const uint16_t* r = pool + sl[k] * IDX_LATENT_RECORD;
            for (int i = 0; i < 4; ++i) o[i] = fmaf(pr[k], bf(r[tid + i * kTile]), o[i]);
        }
    }
    const float inv = m == -INFINITY ? 0.0f : 1.0f / l;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + (row * a.heads + h) * IDX_LATENT_DIM;
    for (int i = 0; i < 4; ++i) out[tid + i * kTile] = __float2bfloat16_rn(o[i] * inv);
    if (a.lse != nullptr && tid == 0) a.lse[row * a.heads + h] = m == -INFINITY ? -INFINITY : m + logf(l);
}

}  // namespace

size_t attend_ws_bytes(int64_t, int, int64_t) { return 256; }

cudaError_t launch_attend(const AttendArgs& a, int sms, cudaStream_t st) {
    (void)sms;
    attend_kernel<<<dim3(static_cast<unsigned>(a.rows), a.heads, 1), kTile, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace dsaidx
