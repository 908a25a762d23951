// qlatent_append.cu -- idx_qlatent_append and idx_qlatent_read: a token's latent
// vector and its turned position part into a record in 8 bits, and back.
//
// scale = 2^e, e the least integer with max |latent| <= 448 2^e (448, the
// largest e4m3 number, is 1.75 2^8): the exponent of the largest magnitude less
// 8, and one more where its fraction passes 0.75.  Division by a power of two
// is exact, so each latent is rounded once, to its code, and the position part
// keeps the bf16 that the bf16 cache would hold.
//
// Bound by memory: 1152 bytes on one side and 644 on the other, a token.  A warp
// a token, 16 latents (one 16-byte vector of codes) and a pair of position
// elements a lane, four tokens a CTA, so that a decode step's few tokens still
// spread over many SMs.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "latent_mma.cuh"
#include "qlatent.h"
#include "rope.cuh"

namespace dsaidx {

namespace {

constexpr int kTokensPerCta = 4;
constexpr int kMinExp = -32, kMaxExp = 120;

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
// Two values to e4m3 (nearest even; NaN stays NaN), lo in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t v) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(v)));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// The larger magnitude of the two halves of w and of m, as bf16 bits without
// sign; non-finite ones do not count.
__device__ __forceinline__ uint32_t larger(uint32_t m, uint32_t w) {
    const uint32_t a = w & 0x7FFFu, b = (w >> 16) & 0x7FFFu;
    return max(m, max(a < 0x7F80u ? a : 0u, b < 0x7F80u ? b : 0u));
}

// Where a record and its scale are; false where the slot names none.
__device__ __forceinline__ bool record_at(int64_t slot, int64_t num_slots, int block_size, int64_t block_bytes,
                                          int32_t* status, int64_t& row, int64_t& scale) {
    if (slot < 0) return false;
    if (slot >= num_slots) {
        if (lane_id() == 0) set_status(status, IDX_ERR_DEVICE_CHECK);
        return false;
    }
    const int s = static_cast<int>(slot), b = s / block_size, o = s - b * block_size;
    row = b * block_bytes + static_cast<int64_t>(o) * kQRow;
    scale = b * block_bytes + static_cast<int64_t>(block_size) * kQRow + 4 * o;
    return true;
}

__global__ void __launch_bounds__(32 * kTokensPerCta) qappend_kernel(const QAppendArgs q) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const AppendArgs& a = q.a;
    const int lane = lane_id();
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kTokensPerCta + warp_id();
    if (t >= a.n) return;
    // slot, latents and position part in flight together
    const int64_t slot = a.slots[t];
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.latent) + t * a.latent_stride);
    const uint4 u = src[2 * lane], v = src[2 * lane + 1];
    const uint32_t* pe = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.pe) + t * a.pe_stride);
    uint32_t p = pe[lane];
    int64_t row, at;
    if (!record_at(slot, a.num_slots, q.block_size, q.block_bytes, a.status, row, at)) return;
    const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = larger(top, w[i]);
    top = __reduce_max_sync(~0u, top);
    int e = static_cast<int>(top >> 7) - 127 - 8 + ((top & 127u) > 96u ? 1 : 0);
    e = top == 0u ? 0 : min(max(e, kMinExp), kMaxExp);
    const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float x[4] = {bf_lo(w[2 * i]), bf_hi(w[2 * i]), bf_lo(w[2 * i + 1]), bf_hi(w[2 * i + 1])};
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = (x[k] - x[k] == 0.0f ? x[k] : __uint_as_float(0x7FFFFFFFu)) * inv;
        c[i] = e4m3x2(x[0], x[1]) | e4m3x2(x[2], x[3]) << 16;
    }
    if (a.steps != nullptr) {
        const int64_t pos = a.positions[t];
        float y0, y1;
        if (a.flags & IDX_ROPE_HALF) {
            // elements 2 L and 2 L + 1 of the first half pair with those 32 further on
            const uint32_t o = pe[lane ^ 16];
            const int first = 2 * (lane & 15);
            const float2 c0 = rope_cs(pos, a.steps[first], a.amplitude), c1 = rope_cs(pos, a.steps[first + 1], a.amplitude);
            y0 = lane < 16 ? rope_turn(bf_lo(p), bf_lo(o), c0).x : rope_turn(bf_lo(o), bf_lo(p), c0).y;
            y1 = lane < 16 ? rope_turn(bf_hi(p), bf_hi(o), c1).x : rope_turn(bf_hi(o), bf_hi(p), c1).y;
        } else {
            const float2 y = rope_turn(bf_lo(p), bf_hi(p), rope_cs(pos, a.steps[lane], a.amplitude));
            y0 = y.x;
            y1 = y.y;
        }
        p = bf16x2(y0, y1);
    }
    p = bf16x2(bf_lo(p) * inv, bf_hi(p) * inv);
    uint8_t* dst = static_cast<uint8_t*>(a.pool) + row;
    reinterpret_cast<uint4*>(dst)[lane] = make_uint4(c[0], c[1], c[2], c[3]);
    reinterpret_cast<uint32_t*>(dst + kQCodes)[lane] = p;
    if (lane == 0) *reinterpret_cast<float*>(static_cast<uint8_t*>(a.pool) + at) = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}

__global__ void __launch_bounds__(32 * kTokensPerCta) qread_kernel(const QReadArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = lane_id();
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kTokensPerCta + warp_id();
    if (t >= a.n) return;
    uint16_t* dst = static_cast<uint16_t*>(a.out) + t * a.out_stride;
    uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
    uint32_t p = 0u;
    int64_t row, at;
    if (record_at(a.slots[t], a.num_slots, a.block_size, a.block_bytes, a.status, row, at)) {
        const uint8_t* src = static_cast<const uint8_t*>(a.pool);
        const uint4 c = reinterpret_cast<const uint4*>(src + row)[lane];
        const uint32_t pe = reinterpret_cast<const uint32_t*>(src + row + kQCodes)[lane];
        const float s = *reinterpret_cast<const float*>(src + at);
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
        uint32_t r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 x = from_e4m3x2(w[i / 2] >> (16 * (i & 1)) & 0xFFFFu);
            r[i] = bf16x2(x.x * s, x.y * s);
        }
        lo = make_uint4(r[0], r[1], r[2], r[3]);
        hi = make_uint4(r[4], r[5], r[6], r[7]);
        p = bf16x2(bf_lo(pe) * s, bf_hi(pe) * s);
    }
    reinterpret_cast<uint4*>(dst)[2 * lane] = lo;
    reinterpret_cast<uint4*>(dst)[2 * lane + 1] = hi;
    reinterpret_cast<uint32_t*>(dst + IDX_LATENT_DIM)[lane] = p;
}

template <class Args>
cudaError_t launch(void (*kernel)(Args), int64_t n, const Args& a, cudaStream_t st) {
    const int64_t grid = (n + kTokensPerCta - 1) / kTokensPerCta;
    if (grid >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(32 * kTokensPerCta, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_qappend(const QAppendArgs& a, cudaStream_t st) { return launch(qappend_kernel, a.a.n, a, st); }
cudaError_t launch_qread(const QReadArgs& a, cudaStream_t st) { return launch(qread_kernel, a.n, a, st); }

}  // namespace dsaidx
