// rope.cu -- idx_rope: rotary positions on part of every head.
//
// Bound by memory: each element is read and written once.  A CTA takes a run
// of (token, head) rows, computes the cosines and sines of the tokens it spans
// once into shared memory (one integer multiply and one sincospi a pair,
// shared by all heads of a token) and turns the rows with up to 16-byte
// accesses, kRows rows in flight a thread.  Block shape: x covers the work
// items of one row (a vector of kVec elements; with pairs half a head apart,
// a vector and its partner together, so that a turn in place has one owner),
// y the rows, so only the token of a row takes a division.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "latent.h"
#include "rope.cuh"

namespace dsaidx {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeRows = 4;              // rows in flight a thread
constexpr int kRopeTableBytes = 40960;    // cosines and sines of the tokens a CTA spans

template <class T> __device__ __forceinline__ float to_f32(T v) { return static_cast<float>(v); }
template <class T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <class T, int kVec>
struct alignas(sizeof(T) * kVec) Vec {
    T v[kVec];
};

struct RopeParams {
    const void* x;
    void* y;
    const int64_t* pos;
    const uint64_t* steps;
    int64_t xt, xh, yt, yh, rows;
    int heads, head_dim, rot, offset, rows_per_cta, items;
    int rot_items;      // of the items: rotated ones first, then copies
    int step, dist;     // split pairs: elements from item to item, from a to b
    float amplitude;
    float sign;         // -1: the transposed map
};

// kSplit: a pair's two values lie in two vectors (halves; or interleaved pairs
// that no two-element access may touch); else next to each other in one.
template <class T, int kVec, bool kSplit>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
    extern __shared__ float2 cs[];   // [tokens spanned][rot / 2]
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int np = p.rot >> 1;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * p.rows_per_cta;
    const int rows = static_cast<int>(p.rows - row0 < p.rows_per_cta ? p.rows - row0 : p.rows_per_cta);
    const int64_t t0 = row0 / p.heads;
    const int h0 = static_cast<int>(row0 - t0 * p.heads);
    const int toks = (h0 + rows - 1) / p.heads + 1;
    const int tid = threadIdx.y * blockDim.x + threadIdx.x, nthr = blockDim.x * blockDim.y;
    for (int i = tid; i < toks * np; i += nthr) {
        const int t = i / np, k = i - t * np;
        float2 v = rope_cs(p.pos[t0 + t], p.steps[k], p.amplitude);
        v.y *= p.sign;
        cs[i] = v;
    }
    __syncthreads();
    using V = Vec<T, kVec>;
    for (int item = threadIdx.x; item < p.items; item += blockDim.x) {
        const bool turned = item < p.rot_items;
        // element of the head this item starts at, and its first pair
        int e, pair = 0;
        if (turned) {
            e = p.offset + item * (kSplit ? p.step : kVec);
            pair = kSplit ? item * kVec : item * kVec / 2;
        } else {
            e = (item - p.rot_items) * kVec;
            if (e >= p.offset) e += p.rot;
        }
        for (int r0 = threadIdx.y; r0 < rows; r0 += kRopeRows * blockDim.y) {
            V a[kRopeRows], b[kRopeRows];
            int t[kRopeRows], h[kRopeRows];
#pragma unroll
            for (int u = 0; u < kRopeRows; ++u) {
                const int r = r0 + u * blockDim.y;
                if (r >= rows) continue;
                t[u] = (h0 + r) / p.heads;
                h[u] = h0 + r - t[u] * p.heads;
                const T* src = static_cast<const T*>(p.x) + (t0 + t[u]) * p.xt + h[u] * p.xh + e;
                a[u] = *reinterpret_cast<const V*>(src);
                if constexpr (kSplit)
                    if (turned) b[u] = *reinterpret_cast<const V*>(src + p.dist);
            }
#pragma unroll
            for (int u = 0; u < kRopeRows; ++u) {
                const int r = r0 + u * blockDim.y;
                if (r >= rows) continue;
                T* dst = static_cast<T*>(p.y) + (t0 + t[u]) * p.yt + h[u] * p.yh + e;
                if (turned) {
                    const float2* c = cs + t[u] * np + pair;
                    if constexpr (kSplit) {
#pragma unroll
                        for (int j = 0; j < kVec; ++j) {
                            const float2 o = rope_turn(to_f32(a[u].v[j]), to_f32(b[u].v[j]), c[j]);
                            a[u].v[j] = from_f32<T>(o.x);
                            b[u].v[j] = from_f32<T>(o.y);
                        }
                        *reinterpret_cast<V*>(dst + p.dist) = b[u];
                    } else {
#pragma unroll
                        for (int j = 0; j < kVec / 2; ++j) {
                            const float2 o = rope_turn(to_f32(a[u].v[2 * j]), to_f32(a[u].v[2 * j + 1]), c[j]);
                            a[u].v[2 * j] = from_f32<T>(o.x);
                            a[u].v[2 * j + 1] = from_f32<T>(o.y);
                        }
                    }
                }
                *reinterpret_cast<V*>(dst) = a[u];
            }
        }
    }
}

template <class T, int kVec, bool kSplit>
cudaError_t launch_rope_t(RopeParams p, bool half, bool inplace, int sms, cudaStream_t st) {
    p.step = half ? kVec : 2;
    p.dist = half ? p.rot / 2 : 1;
    p.rot_items = kSplit ? p.rot / 2 / kVec : p.rot / kVec;
    p.items = p.rot_items + (inplace ? 0 : (p.head_dim - p.rot) / kVec);
    const int bx = p.items < kRopeThreads ? p.items : kRopeThreads, by = kRopeThreads / bx;
    // kRopeRows rows a thread where that leaves two CTAs an SM, else one; the
    // table of the tokens spanned (rows / heads + 2 at most) has to fit
    int64_t rpc = static_cast<int64_t>(kRopeRows) * by;
    if ((p.rows + rpc - 1) / rpc < 2 * sms) rpc = by;
    const int fit = kRopeTableBytes / (p.rot / 2 * 8);   // >= 10 tokens
    if (rpc / p.heads + 2 > fit) rpc = static_cast<int64_t>(fit - 2) * p.heads;
    p.rows_per_cta = static_cast<int>(rpc);
    const int64_t toks = rpc / p.heads + 2;
    const int64_t grid = (p.rows + rpc - 1) / rpc;
    if (grid >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(bx), static_cast<unsigned>(by), 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(toks) * (p.rot / 2) * 8;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rope_kernel<T, kVec, kSplit>, p);
}

// Elements of the widest access (16 bytes at most) that every address it is
// made at is a multiple of.
int vec_of(const RopeParams& p, int esize, bool half) {
    int v = 16 / esize;
    const uintptr_t base = reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.y);
    const int64_t elems = p.xt | p.xh | p.yt | p.yh | p.offset | p.head_dim | (half ? p.rot / 2 : p.rot);
    while (v > 1 && (base % (static_cast<uintptr_t>(v) * esize) != 0 || elems % v != 0)) v /= 2;
    return v;
}

template <class T>
cudaError_t launch_rope_dt(const RopeParams& p, bool half, bool inplace, int sms, cudaStream_t st) {
    const int v = vec_of(p, sizeof(T), half);
    if constexpr (sizeof(T) == 2)
        if (v == 8)
            return half ? launch_rope_t<T, 8, true>(p, half, inplace, sms, st)
                        : launch_rope_t<T, 8, false>(p, half, inplace, sms, st);
    if (v == 4)
        return half ? launch_rope_t<T, 4, true>(p, half, inplace, sms, st)
                    : launch_rope_t<T, 4, false>(p, half, inplace, sms, st);
    if (v == 2)
        return half ? launch_rope_t<T, 2, true>(p, half, inplace, sms, st)
                    : launch_rope_t<T, 2, false>(p, half, inplace, sms, st);
    return launch_rope_t<T, 1, true>(p, half, inplace, sms, st);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int sms, cudaStream_t st) {
    RopeParams p{};
    p.x = a.x; p.y = a.y; p.pos = a.positions; p.steps = a.steps;
    p.xt = a.xt; p.xh = a.xh; p.yt = a.yt; p.yh = a.yh;
    p.rows = a.tokens * a.heads;
    p.heads = a.heads; p.head_dim = a.head_dim; p.rot = a.rot; p.offset = a.offset;
    p.amplitude = a.amplitude;
    p.sign = (a.flags & IDX_ROPE_TRANSPOSE) ? -1.0f : 1.0f;
    const bool half = (a.flags & IDX_ROPE_HALF) != 0, inplace = a.x == a.y;
    if (a.dtype == IDX_DT_BF16) return launch_rope_dt<__nv_bfloat16>(p, half, inplace, sms, st);
    if (a.dtype == IDX_DT_FP16) return launch_rope_dt<__half>(p, half, inplace, sms, st);
    return launch_rope_dt<float>(p, half, inplace, sms, st);
}

}  // namespace dsaidx
