// rope.cu -- idx_rope: rotary positions on part of every head.
//
// Bound by memory: each element is read and written once, so everything else
// is kept off the path.  A CTA takes the heads of one token, or of several
// where there are few heads; a thread takes one work item of a head (a vector
// of up to 16 bytes; with pairs half a head apart a vector and its partner
// together, so that a turn in place has one owner) and keeps it and its token
// over all its heads, so its addresses advance by one stride; the CTA computes
// each pair's cosine and sine once (one integer multiply and one sincospi),
// while the first heads' values are on their way.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "latent.h"
#include "rope.cuh"

namespace dsaidx {

namespace {

// Most threads of a CTA.  8192 x 64 heads x 128, half of each turned in halves:
// 49 us (5.5 TB/s); with 256 (192 used) some 7 % more, 4000 x 64 x 192
// interleaved 40 us against 36.
constexpr int kRopeThreads = 128;

template <class T> __device__ __forceinline__ float to_f32(T v) { return static_cast<float>(v); }
template <class T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <class T, int kVec>
struct alignas(sizeof(T) * kVec) Vec {
    T v[kVec];
};

// A pair's cosine and sine, read each time: kept in registers over the heads
// they cost 16 of them, and with them loads in flight (8192 x 64 heads x 128,
// half turned in halves: 49 us, 52 from registers).
__device__ __forceinline__ float2 table(const float2* p) {
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(smem_u32(p)) : "memory");
    return v;
}

struct RopeParams {
    const void* x;
    void* y;
    const int64_t* pos;
    const uint64_t* steps;
    int64_t xt, xh, yt, yh, tokens;
    int heads, head_dim, rot, offset, items;
    int rot_items;         // of the items: rotated ones first, then copies
    int step, dist;        // split pairs: elements from item to item, from a to b
    int tok_cta, hy;       // tokens a CTA, heads of a token taken at once
    int heads_cta;         // heads a CTA (blockIdx.y)
    float amplitude;
    float sign;            // -1: the transposed map
};

// kSplit: a pair's two values lie in two vectors (halves; or interleaved pairs
// that no two-element access may touch); else next to each other in one.
template <class T, int kVec, bool kSplit>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
    extern __shared__ float2 cs[];   // [tok_cta][rot / 2]
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    using V = Vec<T, kVec>;
    constexpr int kPairs = kSplit ? kVec : kVec / 2;
    // heads in flight a thread; two vectors of a split pair are enough (two
    // heads of them: 53 us in the case above, for want of registers)
    constexpr int kRopeHeads = kSplit ? 1 : 2;
    const int np = p.rot >> 1;
    const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * p.tok_cta;
    const int toks = static_cast<int>(p.tokens - tok0 < p.tok_cta ? p.tokens - tok0 : p.tok_cta);
    // item and head of this thread: the rotated items of all heads first, so
    // that few warps hold both kinds
    int item = threadIdx.x, ty = 0;
    if (p.items <= kRopeThreads) {
        const int first = p.rot_items * p.hy * p.tok_cta;
        const bool copies = item >= first;
        const int n = copies ? p.items - p.rot_items : p.rot_items, i = copies ? item - first : item;
        ty = i / n;
        item = i - ty * n + (copies ? p.rot_items : 0);
    }
    const int tl = ty / p.hy;
    const int h0 = blockIdx.y * p.heads_cta + ty - tl * p.hy;
    const int h1 = tl < toks ? min(p.heads, (static_cast<int>(blockIdx.y) + 1) * p.heads_cta) : 0;
    const T* x = static_cast<const T*>(p.x) + (tok0 + tl) * p.xt;
    T* y = static_cast<T*>(p.y) + (tok0 + tl) * p.yt;
    V a[kRopeHeads], b[kRopeHeads];
    bool turned = false;
    int e = 0;                       // element of the head the item starts at
    auto load = [&](int item, int h) {
        turned = item < p.rot_items;
        if (turned) {
            e = p.offset + item * (kSplit ? p.step : kVec);
        } else {
            e = (item - p.rot_items) * kVec;
            if (e >= p.offset) e += p.rot;
        }
#pragma unroll
        for (int u = 0; u < kRopeHeads; ++u) {
            if (h + u * p.hy >= h1) continue;
            const T* src = x + (h + u * p.hy) * p.xh + e;
            a[u] = *reinterpret_cast<const V*>(src);
            if constexpr (kSplit)
                if (turned) b[u] = *reinterpret_cast<const V*>(src + p.dist);
        }
    };
    // the first values are on their way while the table is made
    load(item, h0);
    for (int i = threadIdx.x; i < toks * np; i += blockDim.x) {
        const int tk = i / np, k = i - tk * np;
        float2 v = rope_cs(p.pos[tok0 + tk], p.steps[k], p.amplitude);
        v.y *= p.sign;
        cs[i] = v;
    }
    __syncthreads();
    while (true) {
        const float2* c = cs + tl * np + item * kPairs;
        for (int h = h0; h < h1; h += kRopeHeads * p.hy) {
            if (h != h0) load(item, h);
#pragma unroll
            for (int u = 0; u < kRopeHeads; ++u) {
                if (h + u * p.hy >= h1) continue;
                T* dst = y + (h + u * p.hy) * p.yh + e;
                if (turned) {
                    if constexpr (kSplit) {
#pragma unroll
                        for (int j = 0; j < kVec; ++j) {
                            const float2 o = rope_turn(to_f32(a[u].v[j]), to_f32(b[u].v[j]), table(c + j));
                            a[u].v[j] = from_f32<T>(o.x);
                            b[u].v[j] = from_f32<T>(o.y);
                        }
                        *reinterpret_cast<V*>(dst + p.dist) = b[u];
                    } else {
#pragma unroll
                        for (int j = 0; j < kVec / 2; ++j) {
                            const float2 o = rope_turn(to_f32(a[u].v[2 * j]), to_f32(a[u].v[2 * j + 1]), table(c + j));
                            a[u].v[2 * j] = from_f32<T>(o.x);
                            a[u].v[2 * j + 1] = from_f32<T>(o.y);
                        }
                    }
                }
                *reinterpret_cast<V*>(dst) = a[u];
            }
        }
        item += kRopeThreads;            // a head of more items than threads
        if (item >= p.items) break;
        load(item, h0);
    }
}

template <class T, int kVec, bool kSplit>
cudaError_t launch_rope_t(RopeParams p, bool half, bool inplace, int sms, cudaStream_t st) {
    p.step = half ? kVec : 2;
    p.dist = half ? p.rot / 2 : 1;
    p.rot_items = kSplit ? p.rot / 2 / kVec : p.rot / kVec;
    p.items = p.rot_items + (inplace ? 0 : (p.head_dim - p.rot) / kVec);
    const int most = p.items < kRopeThreads ? kRopeThreads / p.items : 1;
    // the heads of a token in rounds of hy, or several tokens' heads: the largest
    // hy that leaves the fewest threads idle in the last round, not below two
    // thirds of the CTA (64 heads of 12 items: 8 rounds of 8 heads take 8 %
    // less than 7 of 10)
    p.hy = p.heads < most ? p.heads : most;
    for (int hy = p.hy - 1; hy >= 1 && 3 * hy >= 2 * most; --hy)
        if ((p.heads + hy - 1) / hy * hy < (p.heads + p.hy - 1) / p.hy * p.hy) p.hy = hy;
    const int rounds = (p.heads + p.hy - 1) / p.hy;
    p.tok_cta = most / p.hy;
    if (p.tok_cta > p.tokens) p.tok_cta = static_cast<int>(p.tokens);
    // few tokens: their heads go to several CTAs, down to one round each
    const int64_t groups = (p.tokens + p.tok_cta - 1) / p.tok_cta;
    int64_t splits = (2 * sms + groups - 1) / groups;
    if (splits > rounds) splits = rounds;
    p.heads_cta = static_cast<int>((rounds + splits - 1) / splits) * p.hy;
    if (groups >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(groups), static_cast<unsigned>((p.heads + p.heads_cta - 1) / p.heads_cta), 1);
    const int threads = p.items < kRopeThreads ? p.items * p.hy * p.tok_cta : kRopeThreads;
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(p.tok_cta) * (p.rot / 2) * sizeof(float2);   // at most 16 KB
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
    p.tokens = a.tokens;
    p.heads = a.heads; p.head_dim = a.head_dim; p.rot = a.rot; p.offset = a.offset;
    p.amplitude = a.amplitude;
    p.sign = (a.flags & IDX_ROPE_TRANSPOSE) ? -1.0f : 1.0f;
    const bool half = (a.flags & IDX_ROPE_HALF) != 0, inplace = a.x == a.y;
    if (a.dtype == IDX_DT_BF16) return launch_rope_dt<__nv_bfloat16>(p, half, inplace, sms, st);
    if (a.dtype == IDX_DT_FP16) return launch_rope_dt<__half>(p, half, inplace, sms, st);
    return launch_rope_dt<float>(p, half, inplace, sms, st);
}

}  // namespace dsaidx
