// latent_append.cu -- idx_latent_append: a token's latent vector and its
// turned position part into its slot of the paged latent cache.
//
// Bound by memory: 1152 bytes read and written a token, once.  72 threads a
// token, one 16-byte chunk each (64 of the latent, 8 of the position part),
// so that every access is full and a decode step's few tokens still spread
// over many SMs.  A thread of the position part computes the angles of its
// own 8 elements; with pairs half a head apart it also reads the partner
// chunk.  8192 tokens 4.2 us, 65,536 tokens 32 us (4.8 TB/s); two or four
// tokens a thread measured the same.
#include <cuda_bf16.h>

#include "common.cuh"
#include "latent.h"
#include "rope.cuh"

namespace dsaidx {

namespace {

constexpr int kChunks = IDX_LATENT_RECORD / 8;      // 16-byte chunks of a record
constexpr int kLatentChunks = IDX_LATENT_DIM / 8;
constexpr int kTokensPerCta = 4;

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&r);
}

__global__ void __launch_bounds__(kChunks * kTokensPerCta) append_kernel(const AppendArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int chunk = threadIdx.x, c = chunk - kLatentChunks;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kTokensPerCta + threadIdx.y;
    if (t >= a.n) return;
    const uint4* pe = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.pe) + t * a.pe_stride);
    // slot and chunk in flight together
    const int64_t slot = a.slots[t];
    uint4 v = c < 0 ? reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.latent) + t * a.latent_stride)[chunk] : pe[c];
    if (slot < 0) return;
    if (slot >= a.num_slots) {
        if (chunk == 0) set_status(a.status, IDX_ERR_DEVICE_CHECK);
        return;
    }
    if (c >= 0 && a.steps != nullptr) {
        const int64_t pos = a.positions[t];
        float x[8], y[8];
        unpack8(v, x);
        if (a.flags & IDX_ROPE_HALF) {
            // elements 8 (c % 4) .. of the first half pair with those 32 further on
            const int first = 8 * (c & 3);
            float other[8];
            unpack8(pe[c ^ 4], other);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 cs = rope_cs(pos, a.steps[first + j], a.amplitude);
                y[j] = c < 4 ? rope_turn(x[j], other[j], cs).x : rope_turn(other[j], x[j], cs).y;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 o = rope_turn(x[2 * j], x[2 * j + 1], rope_cs(pos, a.steps[4 * c + j], a.amplitude));
                y[2 * j] = o.x;
                y[2 * j + 1] = o.y;
            }
        }
        v = make_uint4(pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7]));
    }
    reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.pool) + slot * IDX_LATENT_RECORD)[chunk] = v;
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, cudaStream_t st) {
    const int64_t grid = (a.n + kTokensPerCta - 1) / kTokensPerCta;
    if (grid >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(kChunks, kTokensPerCta, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, append_kernel, a);
}

}  // namespace dsaidx
