// latent_rows.cuh -- what the absorbed attention kernels share: the keys of a
// row, how rows are spread over CTAs (whole, cut into equal runs of the line of
// all tiles, or over a cluster) and the join of the rows that were cut.
#pragma once

#include <cuda_bf16.h>

#include "internal.h"
#include "latent.h"
#include "latent_mma.cuh"

namespace dsaidx {

namespace {

constexpr int kMaxCtas = 152;              // one an SM; CTAs of different clusters never wait on one another
constexpr int kMinRun = 2;                 // tiles a CTA, at least, where rows are cut
constexpr float kNone = -3.0e38f;          // maximum of a head without a key so far

// What the rows of a call are and where their results go.
struct RowParams {
    const int64_t* slots;
    int64_t slots_stride;
    const int32_t* block_table;
    const int32_t* seq_lens;
    int64_t rows, num_slots;
    int block_size, mbps, heads, hgs, max_keys;
    int split;                 // 0: whole rows; 1: the tiles of all rows in equal runs; 2: a row's tiles over a cluster
    const uint8_t* pool;
    float scale_log2;
    __nv_bfloat16* out;
    float* lse;
    int32_t* status;
    float* part_o;             // [2 ctas][N][512]
    float2* part_ml;           // [2 ctas][N]
};

// Visible keys of a row: its length where that is in range, else 0.
__device__ __forceinline__ int row_keys(const RowParams& p, int64_t row) {
    if (p.block_table == nullptr) return p.max_keys;
    const int n = __ldg(p.seq_lens + row);
    if (n < 0 || n > p.max_keys || n > static_cast<int64_t>(p.mbps) * p.block_size) return 0;
    return n;
}
// Tiles (of kTile keys) of a row; one for an empty row, which still writes its result.
template <int kTile>
__device__ __forceinline__ int tiles_of(int keys) { return keys > 0 ? (keys - 1) / kTile + 1 : 1; }

// Where the run of CTA c of g begins in the line of tt tiles.
__device__ __forceinline__ int64_t run_start(int64_t c, int64_t g, int64_t tt) { return c * tt / g; }

// Row in whose tiles position x of the line lies, and where the row begins
// (both scaled by the head groups); with x < 0 the length of the line.
// Executed by a whole warp; paged contexts only.
template <int kTile>
__device__ __forceinline__ void find_row(const RowParams& p, int64_t x, int64_t& row, int64_t& base) {
    const int lane = lane_id();
    int64_t acc = 0;
    for (int64_t r0 = 0; r0 < p.rows; r0 += 32) {
        const int64_t r = r0 + lane;
        int64_t v = r < p.rows ? static_cast<int64_t>(tiles_of<kTile>(row_keys(p, r))) * p.hgs : 0;
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t u = __shfl_up_sync(~0u, v, d);
            if (lane >= d) v += u;
        }
        const unsigned in = __ballot_sync(~0u, x >= 0 && x < acc + v && r < p.rows);
        if (in) {
            const int k = __ffs(in) - 1;
            const int64_t before = __shfl_sync(~0u, v, k > 0 ? k - 1 : 0);
            row = r0 + k;
            base = acc + (k > 0 ? before : 0);
            return;
        }
        acc += __shfl_sync(~0u, v, 31);
    }
    row = p.rows;
    base = acc;
}

// The run [start, end) of CTA c of g in the line of all tiles, and the row it
// begins in (paged contexts).  A whole warp.  The lengths of up to 32 rows are
// read once.
template <int kTile>
__device__ __forceinline__ void find_run(const RowParams& p, uint32_t c, uint32_t g, int64_t& start, int64_t& end, int64_t& row, int64_t& base) {
    int64_t tt, v = 0;
    if (p.block_table == nullptr) {
        tt = p.rows * p.hgs * tiles_of<kTile>(p.max_keys);
    } else if (p.rows <= 32) {
        const int lane = lane_id();
        // (32 rows of fewer than 2^25 tiles)
        uint32_t n = lane < p.rows ? static_cast<uint32_t>(tiles_of<kTile>(row_keys(p, lane))) : 0u;
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t u = __shfl_up_sync(~0u, n, d);
            if (lane >= d) n += u;
        }
        v = static_cast<int64_t>(n) * p.hgs;
        tt = __shfl_sync(~0u, v, 31);
    } else {
        int64_t none;
        find_row<kTile>(p, -1, none, tt);
    }
    if (tt >> 32 == 0) {      // c tt / g without a long division
        const uint32_t q = static_cast<uint32_t>(tt) / g, r = static_cast<uint32_t>(tt) - q * g;
        start = static_cast<int64_t>(c) * q + c * r / g;
        end = static_cast<int64_t>(c + 1) * q + (c + 1) * r / g;
    } else {
        start = run_start(c, g, tt);
        end = run_start(c + 1, g, tt);
    }
    if (p.block_table == nullptr || start >= end) return;
    if (p.rows > 32) {
        find_row<kTile>(p, start, row, base);
        return;
    }
    const int k = __ffs(__ballot_sync(~0u, start < v)) - 1;      // (lanes behind the last row have its v)
    const int64_t before = __shfl_sync(~0u, v, k > 0 ? k - 1 : 0);
    row = k;
    base = k > 0 ? before : 0;
}

// One piece of work: tiles [t0, t1) of a row's head group.
struct Work {
    int64_t row;
    int hg, keys, t0, t1;
    int slot;       // where its partial sums go; -1: it has all tiles, write the result; -2: the cluster joins
};

// a / b, without a long division where a has 32 bits; both positive.
__device__ __forceinline__ int64_t quotient(int64_t a, int b) {
    return a >> 32 == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
}

// The pieces of this CTA, in order; every role walks them by itself.
template <int kTile>
struct Walk {
    int64_t pos, end;        // split: the run left; whole: item and number of items
    int64_t row, base;       // split, paged: current row and where it begins; cluster: row and head group
    bool first;
    __device__ __forceinline__ Walk(const RowParams& p, int64_t start, int64_t end_, int64_t row_, int64_t base_)
        : pos(start), end(end_), row(row_), base(base_), first(true) {}
    __device__ __forceinline__ bool next(const RowParams& p, Work& w) {
        if (pos >= end) return false;
        if (p.split == 2) {
            w.row = row;
            w.hg = static_cast<int>(base);
            w.keys = row_keys(p, row);
            w.t0 = static_cast<int>(pos);
            w.t1 = static_cast<int>(end);
            w.slot = -2;
            pos = end;
            return true;
        }
        if (!p.split) {
            const uint32_t item = static_cast<uint32_t>(pos), r = item / p.hgs;      // fewer than 2^31 items
            w.row = r;
            w.hg = static_cast<int>(item - r * p.hgs);
            w.keys = row_keys(p, w.row);
            w.t0 = 0;
            w.t1 = tiles_of<kTile>(w.keys);
            w.slot = -1;
            pos += gridDim.x;
            return true;
        }
        int64_t in;
        int nt;
        if (p.block_table == nullptr) {
            w.keys = p.max_keys;
            nt = tiles_of<kTile>(w.keys);
            const int64_t item = quotient(pos, nt);
            w.row = quotient(item, p.hgs);
            w.hg = static_cast<int>(item - w.row * p.hgs);
            in = pos - item * nt;
        } else {
            w.keys = row_keys(p, row);
            nt = tiles_of<kTile>(w.keys);
            if (pos - base >= static_cast<int64_t>(nt) * p.hgs) {
                base += static_cast<int64_t>(nt) * p.hgs;
                ++row;
                w.keys = row_keys(p, row);
                nt = tiles_of<kTile>(w.keys);
            }
            w.row = row;
            w.hg = static_cast<int>(static_cast<uint32_t>(pos - base) / nt);      // (fewer than 2^31 tiles a row)
            in = pos - base - static_cast<int64_t>(w.hg) * nt;
        }
        w.t0 = static_cast<int>(in);
        const int64_t left = end - pos;
        w.t1 = nt - in <= left ? nt : static_cast<int>(in + left);
        w.slot = (w.t0 == 0 && w.t1 == nt) ? -1 : 2 * static_cast<int>(blockIdx.x) + (first ? 0 : 1);
        first = false;
        pos += w.t1 - w.t0;
        return true;
    }
};

// What names key j of a row: its entry of the slot list or of the block table.
// Read a tile ahead; key_slot, which looks at it, comes when it has arrived.
__device__ __forceinline__ int64_t key_entry(const RowParams& p, int64_t row, int keys, int j) {
    if (j >= keys) return -1;
    return p.block_table == nullptr ? __ldg(p.slots + row * p.slots_stride + j)
                                    : static_cast<int64_t>(__ldg(p.block_table + row * p.mbps + j / p.block_size));
}
// Slot of key j; num_slots where it is masked.
__device__ __forceinline__ int key_slot(const RowParams& p, int keys, int j, int64_t entry) {
    const int none = static_cast<int>(p.num_slots);
    if (j >= keys) return none;
    int64_t s = entry;
    if (p.block_table == nullptr) {
        if (s < 0) return none;
    } else {
        s = entry < 0 ? p.num_slots : entry * p.block_size + j % p.block_size;
    }
    if (s >= p.num_slots) {
        set_status(p.status, IDX_ERR_DEVICE_CHECK);
        return none;
    }
    return static_cast<int>(s);
}

// Joins the partial sums of the rows that were cut.  kW warps take the pieces
// of a (row, head) in turn, four of them in flight, lanes over the latent
// dimensions; the warps' sums are added in order.  A CTA has eight warps.
constexpr int kJoinWarps = 8;

template <int kW, int kTile>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const RowParams p, int N, int ctas) {
    __shared__ float acc[kW > 1 ? kJoinWarps : 1][IDX_LATENT_DIM];
    __shared__ float factor[kJoinWarps][kMaxCtas];     // of each piece, 0 where there is nothing
    __shared__ int from[kJoinWarps][kMaxCtas];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t row = blockIdx.x;
    const int warp = warp_id(), lane = lane_id(), wh = warp % kW;
    const int head = blockIdx.y * (kJoinWarps / kW) + warp / kW, hg = head / N, h = head % N;
    const bool live = head < p.heads;
    int64_t a, tt;
    const int nt = tiles_of<kTile>(row_keys(p, row));
    if (p.block_table == nullptr) {
        tt = p.rows * p.hgs * nt;
        a = row * p.hgs * nt;
    } else {
        int64_t before = 0, all = 0;
        for (int64_t r = lane; r < p.rows; r += 32) {
            const int64_t t = static_cast<int64_t>(tiles_of<kTile>(row_keys(p, r))) * p.hgs;
            all += t;
            if (r < row) before += t;
        }
        for (int d = 16; d > 0; d >>= 1) {
            all += __shfl_xor_sync(~0u, all, d);
            before += __shfl_xor_sync(~0u, before, d);
        }
        tt = all;
        a = before;
    }
    a += static_cast<int64_t>(hg) * nt;
    const int64_t b = a + nt;
    // first and last CTA with a tile of [a, b)
    int64_t c0 = a * ctas / tt, c1;
    while (run_start(c0 + 1, ctas, tt) <= a) ++c0;
    c1 = (b - 1) * ctas / tt;
    while (run_start(c1 + 1, ctas, tt) < b) ++c1;
    // (one CTA: it wrote the result.)  A run may be empty; the row is the second
    // piece of its first CTA unless it begins with that CTA's run.
    const bool cut = live && c0 != c1;
    const int pieces = static_cast<int>(c1 - c0) + 1;
    float m = kNone, l = 0.0f;
    float4 o[4] = {};
    if (cut) {
        // every warp looks the pieces up, a lane a piece
        constexpr int kRounds = (kMaxCtas + 31) / 32;
        float2 ml[kRounds];
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const int k = 32 * r + lane;
            ml[r] = make_float2(kNone, 0.0f);
            if (k >= pieces) continue;
            const int64_t start = run_start(c0 + k, ctas, tt);
            const bool empty = start == run_start(c0 + k + 1, ctas, tt);
            const int at = empty ? -1 : static_cast<int>(2 * (c0 + k) + (start < a ? 1 : 0)) * N + h;
            from[warp][k] = at;
            if (!empty) ml[r] = p.part_ml[at];
        }
        __syncwarp();
        // the first pieces' sums are on their way beside their statistics
        float4 v[4][4];
        auto load = [&](int k0) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int k = k0 + u * kW, at = k < pieces ? from[warp][k] : -1;
                if (at < 0) continue;
                const float4* src = reinterpret_cast<const float4*>(p.part_o + static_cast<int64_t>(at) * IDX_LATENT_DIM);
#pragma unroll
                for (int q = 0; q < 4; ++q) v[u][q] = __ldg(src + 32 * q + lane);
            }
        };
        load(wh);
#pragma unroll
        for (int r = 0; r < kRounds; ++r)
            if (ml[r].y != 0.0f) m = fmaxf(m, ml[r].x);
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const float f = ml[r].y != 0.0f ? exp2_fast(ml[r].x - m) : 0.0f;
            if (f != 0.0f) l += ml[r].y * f;
            if (32 * r + lane < pieces) factor[warp][32 * r + lane] = f;
        }
        for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(~0u, l, d);
        __syncwarp();
        for (int k0 = wh; k0 < pieces; k0 += 4 * kW) {
            if (k0 != wh) load(k0);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int k = k0 + u * kW;
                const float f = k < pieces ? factor[warp][k] : 0.0f;      // (0: there is nothing)
                if (f == 0.0f) continue;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    o[q].x += v[u][q].x * f;
                    o[q].y += v[u][q].y * f;
                    o[q].z += v[u][q].z * f;
                    o[q].w += v[u][q].w * f;
                }
            }
        }
    }
    if constexpr (kW > 1) {
#pragma unroll
        for (int q = 0; q < 4; ++q) reinterpret_cast<float4*>(acc[warp])[32 * q + lane] = o[q];
        __syncthreads();
        if (wh != 0) return;
#pragma unroll
        for (int k = 1; k < kW; ++k) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 v = reinterpret_cast<const float4*>(acc[warp + k])[32 * q + lane];
                o[q].x += v.x;
                o[q].y += v.y;
                o[q].z += v.z;
                o[q].w += v.w;
            }
        }
    }
    if (!cut) return;
    const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
    uint2* out = reinterpret_cast<uint2*>(p.out + (row * p.heads + head) * IDX_LATENT_DIM);
#pragma unroll
    for (int q = 0; q < 4; ++q)
        out[32 * q + lane] = make_uint2(bf16x2(o[q].x * inv, o[q].y * inv), bf16x2(o[q].z * inv, o[q].w * inv));
    if (lane == 0 && p.lse != nullptr)
        p.lse[row * p.heads + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

// Launches the join of a call that was cut over `ctas` CTAs.
template <int kTile>
cudaError_t launch_join(const RowParams& p, int N, int ctas, cudaStream_t st) {
    // warps a (row, head): eight where rows have many pieces, else as many as
    // there is parallelism for.  Measured: 9 rows to 75 pieces, 16 heads, whole
    // call 403 us with one warp, 369 with eight; 32 rows of 3.4 pieces, 128
    // heads, 46 us with one, 57 with four, 74 with eight; 32 rows of 4.8
    // pieces, 16 heads, 58.6, 55.1 and 58.0 us.
    const int warps = ctas > 6 * p.rows * p.hgs ? 8 : p.rows * p.heads <= 1024 ? 4 : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.rows), static_cast<unsigned>((p.heads * warps + kJoinWarps - 1) / kJoinWarps), 1);
    cfg.blockDim = dim3(32 * kJoinWarps, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    kt_mark(st);
    const cudaError_t e =
        cudaLaunchKernelEx(&cfg, warps == 8 ? join_kernel<8, kTile> : warps == 4 ? join_kernel<4, kTile> : join_kernel<1, kTile>, p, N, ctas);
    kt_mark(st);
    return e;
}

// Heads of one score product.
inline int width_of(int heads) { return heads <= 16 ? 16 : heads <= 32 ? 32 : 64; }

// How the rows are spread over CTAs.
struct Shape {
    int N, hgs, split, ctas, cluster;
};

}  // namespace

}  // namespace dsaidx
