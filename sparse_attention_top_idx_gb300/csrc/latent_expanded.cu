// latent_expanded.cu -- expanded causal attention of packed prompts: one CTA a
// (query, head), keys in tiles of 128, one pass with the running maximum and
// sum of the softmax in fp32.
#include <cuda_bf16.h>

#include <cmath>

#include "common.cuh"
#include "latent.h"

namespace dsaidx {

namespace {

constexpr int kTile = 128;
constexpr int kN = IDX_EXPANDED_NOPE_DIM, kP = IDX_LATENT_PE_DIM, kV = IDX_EXPANDED_V_DIM;

__device__ __forceinline__ float bf(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

__global__ void __launch_bounds__(kTile) expanded_kernel(const ExpandedArgs a) {
    __shared__ float q[kN + kP];
    __shared__ float pr[kTile];
    __shared__ float red[4];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t t = blockIdx.x;
    const int h = blockIdx.y, tid = threadIdx.x;
    int b = 0;
    while (b < a.batch && !(t >= a.cu_q[b] && t < a.cu_q[b + 1])) ++b;
    if (b == a.batch) return;
    const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
    if (q0 < 0 || q1 > a.total_q || k0 < 0 || k1 < k0 || k1 > a.total_k) {
        set_status(a.status, IDX_ERR_DEVICE_CHECK);
        return;
    }
    const int n = max(0, (k1 - k0) - (q1 - q0) + static_cast<int>(t - q0) + 1);
    for (int i = tid; i < kN + kP; i += kTile) q[i] = bf(static_cast<const uint16_t*>(a.q)[t * a.q_row + h * a.q_head + i]);
    float m = -INFINITY, l = 0.0f, o = 0.0f;
    for (int j0 = 0; j0 < n; j0 += kTile) {
        __syncthreads();
        float s = -INFINITY;
        if (j0 + tid < n) {
            const int64_t j = k0 + j0 + tid;
            const uint16_t* kn = static_cast<const uint16_t*>(a.kn) + j * a.kn_row + h * a.kn_head;
            const uint16_t* kp = static_cast<const uint16_t*>(a.kp) + j * a.kp_row;
            s = 0.0f;
            for (int i = 0; i < kN; ++i) s = fmaf(q[i], bf(kn[i]), s);
            for (int i = 0; i < kP; ++i) s = fmaf(q[kN + i], bf(kp[i]), s);
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
        pr[tid] = j0 + tid < n ? expf(s - mn) : 0.0f;
        __syncthreads();
        l *= c;
        o *= c;
        for (int k = 0; k < kTile && j0 + k < n; ++k) {
            l += pr[k];
            o = fmaf(pr[k], bf(static_cast<const uint16_t*>(a.v)[(k0 + j0 + k) * a.v_row + h * a.v_head + tid]), o);
        }
    }
    const float inv = m == -INFINITY ? 0.0f : 1.0f / l;
    static_cast<__nv_bfloat16*>(a.out)[(t * a.heads + h) * kV + tid] = __float2bfloat16_rn(o * inv);
    if (a.lse != nullptr && tid == 0) a.lse[t * a.heads + h] = m == -INFINITY ? -INFINITY : m + logf(l);
}

}  // namespace

cudaError_t launch_expanded(const ExpandedArgs& a, int sms, cudaStream_t st) {
    (void)sms;
    expanded_kernel<<<dim3(static_cast<unsigned>(a.total_q), a.heads, 1), kTile, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace dsaidx
