// qlatent_attend.cu -- absorbed latent attention over records in 8 bits.
//
// A CTA a row and 8 heads, a warp a head: tiles of 32 keys are decoded into
// shared memory, lane = key for the scores and lane = 16 latent dimensions for
// the values, with the running maximum and sum of a softmax in fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "latent_rows.cuh"
#include "qlatent.h"

namespace dsaidx {

namespace {

constexpr int kHeadsCta = 8, kTile = 32, kPitch = IDX_LATENT_RECORD + 1;

struct QParams : RowParams {
    const __nv_bfloat16* ql;
    const __nv_bfloat16* qp;
    int64_t ql_row, ql_head, qp_row, qp_head, block_bytes;
};

__global__ void __launch_bounds__(32 * kHeadsCta) qattend_kernel(const QParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    extern __shared__ float sh[];
    float* rec = sh;                                  // [kTile][kPitch]
    float* q = sh + kTile * kPitch;                   // [kHeadsCta][576]
    __shared__ int slots[kTile];
    const int64_t row = blockIdx.x;
    const int warp = warp_id(), lane = lane_id(), head = blockIdx.y * kHeadsCta + warp;
    const int h = min(head, p.heads - 1);
    for (int d = lane; d < IDX_LATENT_RECORD; d += 32)
        q[warp * IDX_LATENT_RECORD + d] = __bfloat162float(
            d < IDX_LATENT_DIM ? p.ql[row * p.ql_row + h * p.ql_head + d]
                               : p.qp[row * p.qp_row + h * p.qp_head + d - IDX_LATENT_DIM]);
    const int keys = row_keys(p, row);
    if (p.block_table != nullptr && keys == 0 && threadIdx.x == 0 && p.seq_lens[row] != 0)
        set_status(p.status, IDX_ERR_DEVICE_CHECK);
    float m = kNone, l = 0.0f, acc[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
    for (int j0 = 0; j0 < keys; j0 += kTile) {
        __syncthreads();
        if (warp == 0) slots[lane] = key_slot(p, keys, j0 + lane, key_entry(p, row, keys, j0 + lane));
        __syncthreads();
        for (int k = warp; k < kTile; k += kHeadsCta) {
            const int s = slots[k];
            if (s == static_cast<int>(p.num_slots)) {
                for (int d = lane; d < IDX_LATENT_RECORD; d += 32) rec[k * kPitch + d] = 0.0f;
                continue;
            }
            const uint8_t* block = p.pool + s / p.block_size * p.block_bytes;
            const uint8_t* src = block + static_cast<int64_t>(s % p.block_size) * kQRow;
            const float scale = *reinterpret_cast<const float*>(block + static_cast<int64_t>(p.block_size) * kQRow + 4 * (s % p.block_size));
            for (int d = 2 * lane; d < IDX_LATENT_DIM; d += 64) {
                uint32_t x;
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(x) : "h"(*reinterpret_cast<const uint16_t*>(src + d)));
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x));
                rec[k * kPitch + d] = f.x * scale;
                rec[k * kPitch + d + 1] = f.y * scale;
            }
            for (int d = lane; d < IDX_LATENT_PE_DIM; d += 32)
                rec[k * kPitch + IDX_LATENT_DIM + d] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(src + kQCodes)[d]) * scale;
        }
        __syncthreads();
        float s = 0.0f;
        for (int d = 0; d < IDX_LATENT_RECORD; ++d) s = fmaf(rec[lane * kPitch + d], q[warp * IDX_LATENT_RECORD + d], s);
        float y = slots[lane] == static_cast<int>(p.num_slots) ? -INFINITY : s * p.scale_log2;
        float top = y;
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
        top = fmaxf(top, m);
        const float f = exp2_fast(m - top), w = exp2_fast(y - top);
        m = top;
        float sum = w;
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
        l = l * f + sum;
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] *= f;
        for (int k = 0; k < kTile; ++k) {
            const float wk = __shfl_sync(~0u, w, k);
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[i] = fmaf(wk, rec[k * kPitch + 32 * i + lane], acc[i]);
        }
    }
    if (head >= p.heads) return;
    const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
    __nv_bfloat16* out = p.out + (row * p.heads + head) * IDX_LATENT_DIM;
#pragma unroll
    for (int i = 0; i < 16; ++i) out[32 * i + lane] = __float2bfloat16_rn(l == 0.0f ? 0.0f : acc[i] * inv);
    if (lane == 0 && p.lse != nullptr)
        p.lse[row * p.heads + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace

size_t qattend_ws_need(int64_t, int, int64_t, bool) { return 256; }

cudaError_t launch_qattend(const AttendArgs& a, int64_t block_bytes, cudaStream_t st) {
    QParams p{};
    p.slots = a.slots; p.slots_stride = a.slots_stride;
    p.block_table = a.block_table; p.seq_lens = a.seq_lens; p.mbps = a.mbps; p.block_size = a.block_size;
    p.pool = static_cast<const uint8_t*>(a.pool);
    p.rows = a.rows; p.num_slots = a.num_slots; p.heads = a.heads; p.max_keys = a.max_keys;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.out = static_cast<__nv_bfloat16*>(a.out); p.lse = a.lse; p.status = a.status;
    p.ql = static_cast<const __nv_bfloat16*>(a.ql); p.qp = static_cast<const __nv_bfloat16*>(a.qp);
    p.ql_row = a.ql_row; p.ql_head = a.ql_head; p.qp_row = a.qp_row; p.qp_head = a.qp_head;
    p.block_bytes = block_bytes;
    static std::atomic<unsigned long long> done{0};
    const int bytes = (kTile * kPitch + kHeadsCta * IDX_LATENT_RECORD) * 4;
    cudaError_t e = set_smem_once(qattend_kernel, bytes, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.rows), static_cast<unsigned>((a.heads + kHeadsCta - 1) / kHeadsCta), 1);
    cfg.blockDim = dim3(32 * kHeadsCta, 1, 1);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    kt_mark(st);
    e = cudaLaunchKernelEx(&cfg, qattend_kernel, p);
    kt_mark(st);
    return e;
}

}  // namespace dsaidx
