// qlatent_attend.cu -- absorbed latent attention over records in 8 bits.
//
// Mathematics, for one row (a query of up to 64 heads) and tiles of 64 keys
// with records s [c | p]:
//   D   = c (q_hi + q_lo / 16) + p q_p      [64 keys, heads]
//   y   = f s D - m,  w = 2^y               f: the head's factor, softmax scale and log2(e)
//   O^T = c^T W,  W = w s 2^11 / s_max      [512, heads]       out = O s_max 2^-11 / sum w
// The codes are operands as they are: nothing is decoded.  What stands on the
// other side is split into 8-bit numbers instead, which is exact or nearly so:
//   queries   a bf16 under a power of two of its head is the sum of two e4m3,
//             the second times 16 (to 2^-22 of the head's largest);
//   weights   9 significant bits are the sum of three e5m2, whose 32 binades
//             hold weights down to 2^-28 of the largest (two e4m3 would hold 8
//             bits down to 2^-9 of it and lose a long context's small weights).
// The parts are further columns of the same product, up to 32 heads: a step
// of 64 keys x 32 columns takes 12.3 ns, of 64 columns 16.4, of 128 columns
// 32.7; of 128 dimensions x 48, 64 and 96 columns 22.6, 24.7 and 28.7.  At 64
// heads three products share the accumulators, as TMEM has no more columns.
// The position part is a bf16 product into the same accumulators, halved, once
// for each half of their columns (0 times an infinite key would be NaN).
//
// One persistent CTA an SM, warp-specialised:
//   warp 0     one lane issues the score products
//   warp 2     one lane issues the value products
//   warps 4-7, at 64 heads 12-15 too  softmax, half of the heads each, and
//              epilogue, half of the dimensions each; a thread has one key
//   warps 8-11 gather records, 16 keys of every tile each, with 16-byte
//              asynchronous copies into a ring of tiles (four chunks of 128
//              codes of 64 keys, one of the position parts), and split a row's
//              queries while its first tiles are on their way
//
// The running maximum of a head moves only when a score passes it by 2^4, so
// most tiles need neither a maximum over keys nor a rescaled accumulator.
// Statistics, sums and accumulators are fp32.  Rows are whole, shared by a
// cluster or cut into equal runs as in latent_rows.cuh.
#include <cuda_fp16.h>

#include <cmath>

#include "latent_rows.cuh"
#include "qlatent.h"

namespace dsaidx {

namespace {

constexpr int kChunk = kKeys * 128;        // bytes of a chunk: 128 codes or 64 bf16 of 64 keys
constexpr int kStage = 5 * kChunk;         // a tile: four chunks of codes, one of position parts
constexpr int kFactors = 3;                // rows whose heads' factors are held: the softmax may be two rows behind
constexpr int halves_of(int N) { return N == 64 ? 2 : 1; }      // softmax warpgroups
constexpr int threads_of(int N) { return 256 + 128 * halves_of(N); }
constexpr int kGatherThreads = 128;
constexpr float kGrow = 4.0f;              // log2 by which a score may pass the maximum
constexpr float kTop = 2048.0f;            // a weight of 1 under the largest scale: 2^4 above it is below fp16's largest

// Shared memory: queries (hi and lo rows), two weight tiles, the ring, then
// scales, factors, statistics, masks and barriers.
struct QPlan {
    int stages, p_bytes, p_off, ring_off, scale_off, factor_off, stat_off, mask_off, bar_off, total;
};
__host__ __device__ constexpr QPlan qplan_of(int N) {
    QPlan p{};
    p.stages = N == 64 ? 3 : 4;
    p.p_bytes = N == 16 ? 4096 : N == 32 ? 8192 : 3 * 4096;
    int o = 5 * 2 * N * 128;
    p.p_off = o;      o += 2 * p.p_bytes;
    p.ring_off = o;   o += p.stages * kStage;
    p.scale_off = o;  o += p.stages * kKeys * 4;
    p.factor_off = o; o += kFactors * N * 4;
    p.stat_off = o;   o += 5 * N * 4 + 16;     // four warps' values and one for all; the warps' largest scales
    p.mask_off = o;   o += p.stages * 8;
    p.bar_off = o;    o += (2 * p.stages + 21) * 8;
    p.total = o;
    return p;
}
static_assert(qplan_of(64).total <= 232448 && qplan_of(32).total <= 232448 && qplan_of(16).total <= 232448,
              "fits one SM's shared memory");
static_assert(qplan_of(64).ring_off % 1024 == 0 && qplan_of(32).ring_off % 1024 == 0 && qplan_of(16).ring_off % 1024 == 0,
              "the swizzle's period");

struct QParams : RowParams {
    const uint16_t* ql;
    const uint16_t* qp;
    int64_t ql_row, ql_head, qp_row, qp_head;
    int64_t block_bytes;
};

// MN-major operand of 64-byte rows with the 64-byte swizzle: rows are the K
// index, 8-row groups 512 bytes apart.
__device__ __forceinline__ uint64_t sdesc_mn_sw64(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(4096 >> 4) << 16;
    d |= static_cast<uint64_t>(512 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(4) << 61;
    return d;
}

// kH columns of 16 rows a warp: lanes 0-15 read columns [c, c + kH), lanes
// 16-31 those kH further on, of row lane % 16.
__device__ __forceinline__ void tmem_ld_halves(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16], 16;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld_halves(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8], 8;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_halves(uint32_t (&r)[16]) { tmem_wait_ld16(r); }
__device__ __forceinline__ void tmem_wait_halves(uint32_t (&r)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                 :
                 : "memory");
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Two fp16 to e4m3 (nearest even), and back.
__device__ __forceinline__ uint32_t e4m3x2(uint32_t h) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
    return r;
}
__device__ __forceinline__ uint32_t from_e4m3x2(uint32_t v) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(v)));
    return h;
}
// Two fp16 rounded to the three significant bits of e5m2, whose codes are the
// upper bytes: the magnitudes' low bytes are rounded to nearest.
__device__ __forceinline__ uint32_t to_e5m2(uint32_t h) { return h + 0x00800080u; }
constexpr uint32_t kUpper = 0xFF00FF00u;

__device__ __forceinline__ void copy4_or_zero(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// Combines v[0..kH) over the 16 lanes of a half warp: halves are exchanged, so
// that lane i is left with element i % kH.
template <int kH, class Op>
__device__ __forceinline__ float over_keys(float (&v)[kH], Op op) {
    const int lane = lane_id();
#pragma unroll
    for (int s = kH / 2; s > 0; s /= 2) {
        const bool up = lane & s;
#pragma unroll
        for (int i = 0; i < s; ++i) {
            const float give = up ? v[i] : v[i + s], keep = up ? v[i + s] : v[i];
            v[i] = op(keep, __shfl_xor_sync(~0u, give, s));
        }
    }
    if (kH < 16) v[0] = op(v[0], __shfl_xor_sync(~0u, v[0], 8));
    return v[0];
}

// Splits one head's query: 16 latent elements a lane (u, v) and a pair of
// position elements (p), for row h of the hi rows and row N + h of the lo rows.
// Returns the factor of its scores.
template <int N>
__device__ __forceinline__ float split_query(uint8_t* q, int h, const uint4& u, const uint4& v, uint32_t p, float scale_log2) {
    const int lane = lane_id();
    const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = __vmaxu2(top, w[i] & 0x7FFF7FFFu);
    top = __reduce_max_sync(~0u, max(top & 0xFFFFu, top >> 16));
    // 2^-a brings the largest to [128, 256); a >= -60, so that the position
    // part stays finite
    const uint32_t e = max(top >> 7, 74u);
    const float down = __uint_as_float((261u - e) << 23);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t a[2], b[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t x = w[2 * i + k];
            const uint32_t f = f16x2(__uint_as_float(x << 16) * down, __uint_as_float(x & 0xFFFF0000u) * down);
            a[k] = e4m3x2(f);
            b[k] = e4m3x2(mul_f16x2(sub_f16x2(f, from_e4m3x2(a[k])), 0x4C004C00u));      // 16
        }
        hi[i] = a[0] | a[1] << 16;
        lo[i] = b[0] | b[1] << 16;
    }
    // lane's 16 bytes: piece lane % 8 of chunk lane / 8
    uint8_t* row = q + (lane >> 3) * (2 * N * 128) + h * 128 + (((lane & 7) ^ (h & 7)) << 4);
    *reinterpret_cast<uint4*>(row) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(row + N * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    // half of the position part in the hi rows, the other half (times 16) in the lo rows
    const float p0 = __uint_as_float(p << 16) * (0.5f * down), p1 = __uint_as_float(p & 0xFFFF0000u) * (0.5f * down);
    uint8_t* pe = q + 4 * (2 * N * 128) + h * 128 + (((lane >> 2) ^ (h & 7)) << 4) + 4 * (lane & 3);
    *reinterpret_cast<uint32_t*>(pe) = bf16x2(p0, p1);
    *reinterpret_cast<uint32_t*>(pe + N * 128) = bf16x2(16.0f * p0, 16.0f * p1);
    return top >= 0x7F80u ? __uint_as_float(0x7FFFFFFFu) : scale_log2 * __uint_as_float((e - 7u) << 23);
}

template <int N, int kCl>
__global__ void __launch_bounds__(threads_of(N), 1) qattend_kernel(const QParams p) {
    constexpr QPlan kPlan = qplan_of(N);
    constexpr int kStages = kPlan.stages;
    constexpr int kHalves = halves_of(N), kSoftThreads = 128 * kHalves, kGroupsM = 4 / kHalves;
    constexpr bool kWide = N == 64;            // the weights' parts share the accumulators
    constexpr int kOCols = kWide ? N : 3 * N;  // accumulator columns of 128 dimensions
    constexpr int kSCol = 4 * kOCols;          // first column behind the accumulators
    constexpr int kH = N / kHalves / 2;        // heads a softmax thread
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + kPlan.bar_off);
    uint64_t* full = bar;                        // [stages]
    uint64_t* empty = full + kStages;            // [stages]
    uint64_t* s_full = empty + kStages;          // [2]
    uint64_t* s_empty = s_full + 2;              // [2]
    uint64_t* p_full = s_full + 4;               // [2]
    uint64_t* pv_done = s_full + 6;              // [2]
    uint64_t* q_full = s_full + 8;
    uint64_t* q_empty = s_full + 9;
    uint64_t* o_empty = s_full + 10;
    uint64_t* drain = s_full + 11;               // [2]
    int64_t* sh_run = reinterpret_cast<int64_t*>(s_full + 13);   // start, end, row, base
    uint32_t* sh_tmem = reinterpret_cast<uint32_t*>(s_full + 17);
    int* sh_abort = reinterpret_cast<int*>(sh_tmem + 1);
    uint16_t* masks = reinterpret_cast<uint16_t*>(smem + kPlan.mask_off);   // [stages][4]: 16 keys each
    float* scales = reinterpret_cast<float*>(smem + kPlan.scale_off);       // [stages][64]
    float* factors = reinterpret_cast<float*>(smem + kPlan.factor_off);     // [kFactors][N]
    float* stat = reinterpret_cast<float*>(smem + kPlan.stat_off);          // [5][N], [4]
    const int warp = warp_id(), lane = lane_id();

    if (warp == 0 && elect_one()) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full + i, kGatherThreads + kGatherThreads / 32);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full + i, 1);
            mbar_init(s_empty + i, kSoftThreads);
            mbar_init(p_full + i, kSoftThreads);
            mbar_init(pv_done + i, 1);
            mbar_init(drain + i, 1);
        }
        mbar_init(q_full, kGatherThreads);
        mbar_init(q_empty, 1);
        mbar_init(o_empty, kSoftThreads);
        *sh_abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(sh_tmem, 512);
        tmem_relinquish();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (warp == 2) {
        int64_t start, end, row = 0, base = 0;
        if (kCl > 1) {
            const int item = blockIdx.x / kCl, rank = blockIdx.x % kCl;
            row = item / p.hgs;
            base = item % p.hgs;
            const int64_t nt = tiles_of(row_keys(p, row));
            start = rank * nt / kCl;
            end = (rank + 1) * nt / kCl;
        } else if (!p.split) {
            start = blockIdx.x;
            end = p.rows * p.hgs;
        } else {
            int64_t tt;
            if (p.block_table == nullptr) {
                tt = p.rows * p.hgs * tiles_of(p.max_keys);
            } else {
                int64_t none;
                find_row(p, -1, none, tt);
            }
            start = run_start(blockIdx.x, gridDim.x, tt);
            end = run_start(blockIdx.x + 1, gridDim.x, tt);
            if (p.block_table != nullptr && start < end) find_row(p, start, row, base);
        }
        if (lane == 0) {
            sh_run[0] = start;
            sh_run[1] = end;
            sh_run[2] = row;
            sh_run[3] = base;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *sh_tmem;
    volatile int* abort_flag = sh_abort;
    Walk walk(p, sh_run[0], sh_run[1], sh_run[2], sh_run[3]);
    Work w;

    if (warp >= 8 && warp < 12) {
        // ---- gather: 16 keys of every tile; a row's queries ----
        // A copy instruction moves 128 bytes of four keys: lane / 8 is the key
        // among them, lane % 8 the 16-byte piece.
        const int wq = warp - 8, sub = lane >> 3, piece = lane & 7;
        const uint32_t even = wq * 2048 + sub * 128 + ((piece ^ sub) << 4), odd = even ^ 64u;   // keys 4 k + sub by k
        const uint32_t ring = smem_u32(smem + kPlan.ring_off), sc_addr = smem_u32(scales);
        const int none = static_cast<int>(p.num_slots), j = 16 * wq + (lane & 15);
        const uint32_t block_units = static_cast<uint32_t>(p.block_bytes / 128);
        uint32_t it = 0, item = 0, st = 0, ph = 1;    // tiles, rows, stage and the parity that frees it
        bool ok = true;
        while (ok && walk.next(p, w)) {
            if (p.block_table != nullptr && w.keys == 0 && lane == 0 && __ldg(p.seq_lens + w.row) != 0)
                set_status(p.status, IDX_ERR_DEVICE_CHECK);
            int64_t entry = key_entry(p, w.row, w.keys, w.t0 * kKeys + j);
            // the queries are split behind the copies of the second tile
            const int split_at = min(w.t0 + 1, w.t1 - 1);
            for (int t = w.t0; t < w.t1; ++t, ++it) {
                const int slot = key_slot(p, w.keys, t * kKeys + j, entry);
                const uint32_t valid = __ballot_sync(~0u, slot != none) & 0xFFFFu;
                // a record begins a multiple of 128 bytes into the pool
                const uint32_t own = slot == none ? 0u : static_cast<uint32_t>(slot);
                const uint32_t block = own / static_cast<uint32_t>(p.block_size), at = own - block * p.block_size;
                const uint32_t unit = block * block_units + at * (kQRow / 128);
                const uint8_t* sc = p.pool + block * p.block_bytes + static_cast<int64_t>(p.block_size) * kQRow + 4 * at;
                const uint8_t* src[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    src[k] = p.pool + static_cast<int64_t>(__shfl_sync(~0u, unit, 4 * k + sub)) * 128 + 16 * piece;
                if (t + 1 < w.t1) entry = key_entry(p, w.row, w.keys, (t + 1) * kKeys + j);
                ok = mbar_wait(empty + st, ph, p.status, abort_flag);
                if (!(ok = __all_sync(~0u, ok))) break;
                const uint32_t dst = ring + st * kStage;
#pragma unroll
                for (int c = 0; c < 5; ++c) {
                    if (valid == 0xFFFFu) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) copy16(dst + c * kChunk + ((k & 1) ? odd : even) + 512 * k, src[k] + 128 * c);
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            copy16_or_zero(dst + c * kChunk + ((k & 1) ? odd : even) + 512 * k, src[k] + 128 * c,
                                           (valid >> (4 * k + sub)) & 1 ? 16 : 0);
                    }
                }
                if (lane < 16) copy4_or_zero(sc_addr + (st * kKeys + j) * 4, sc, slot == none ? 0 : 4);
                if (lane == 0) masks[4 * st + wq] = static_cast<uint16_t>(valid);
                copy_arrive(full + st);
                if (lane == 0) mbar_arrive(full + st);
                if (++st == kStages) st = 0, ph ^= 1;
                if (t != split_at) continue;
                ok = mbar_wait(q_empty, (item & 1) ^ 1, p.status, abort_flag);
                if (!(ok = __all_sync(~0u, ok))) break;
                float* factor = factors + item % kFactors * N;
                const int h0 = w.hg * 64;
#pragma unroll 2
                for (int h = wq; h < N; h += 4) {
                    uint4 u = make_uint4(0u, 0u, 0u, 0u), v = u;
                    uint32_t x = 0u;
                    if (h0 + h < p.heads) {
                        const uint4* lat = reinterpret_cast<const uint4*>(p.ql + w.row * p.ql_row + (h0 + h) * p.ql_head);
                        u = __ldg(lat + 2 * lane);
                        v = __ldg(lat + 2 * lane + 1);
                        x = __ldg(reinterpret_cast<const uint32_t*>(p.qp + w.row * p.qp_row + (h0 + h) * p.qp_head) + lane);
                    }
                    const float f = split_query<N>(smem, h, u, v, x, p.scale_log2);
                    if (lane == 0) factor[h] = f;
                }
                fence_proxy_async_smem();
                mbar_arrive(q_full);
                ++item;
            }
        }
        copy_wait_all();
    } else if (warp == 0) {
        // ---- score products ----
        if (elect_one()) {
            constexpr uint32_t kIdS = idesc_make(true, 64, 2 * N), kIdP = idesc_bf16(64, 2 * N, false, false);
            const uint32_t q_addr = smem_u32(smem), ring = smem_u32(smem + kPlan.ring_off);
            uint32_t it = 0, item = 0, st = 0, ph = 0;
            bool ok = true;
            while (ok && walk.next(p, w)) {
                if (!(ok = mbar_wait(q_full, item & 1, p.status, abort_flag))) break;
                for (int t = w.t0; t < w.t1; ++t, ++it) {
                    const uint32_t d = tmem + kSCol + (it & 1) * 2 * N, tile = ring + st * kStage;
                    // the softmax has read the scores before last
                    if (!(ok = mbar_wait(s_empty + (it & 1), ((it >> 1) & 1) ^ 1, p.status, abort_flag))) break;
                    if (!(ok = mbar_wait(full + st, ph, p.status, abort_flag))) break;
                    // records and queries were written by other threads: order
                    // their writes before the tensor core's reads
                    fence_proxy_async_smem();
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        mma_fp8(d, sdesc_sw128(tile + (k >> 2) * kChunk + 32 * (k & 3)),
                                sdesc_sw128(q_addr + (k >> 2) * 2 * N * 128 + 32 * (k & 3)), kIdS, k != 0);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_bf16(d, sdesc_sw128(tile + 4 * kChunk + 32 * k), sdesc_sw128(q_addr + 8 * N * 128 + 32 * k), kIdP, 1u);
                    mma_commit(s_full + (it & 1));
                    if (t + 1 == w.t1) mma_commit(q_empty);
                    if (++st == kStages) st = 0, ph ^= 1;
                }
                ++item;
            }
            // nothing of this CTA may run on when its shared memory and TMEM go
            mma_commit(drain);
            mbar_wait(drain, 0, p.status, nullptr);
        }
    } else if (warp == 2) {
        // ---- value products ----
        if (elect_one()) {
            // e4m3 x e5m2, both operands MN-major
            constexpr uint32_t kIdO = idesc_make(true, 128, kOCols) | 1u << 10 | 1u << 15 | 1u << 16;
            const uint32_t ring = smem_u32(smem + kPlan.ring_off), p_addr = smem_u32(smem + kPlan.p_off);
            uint32_t it = 0, item = 0, st = 0;
            bool ok = true;
            while (ok && walk.next(p, w)) {
                for (int t = w.t0; t < w.t1; ++t, ++it) {
                    // the weights are there, which the records were before them
                    if (!(ok = mbar_wait(p_full + (it & 1), (it >> 1) & 1, p.status, abort_flag))) break;
                    // the accumulators of the piece before were read
                    if (t == w.t0 && !(ok = mbar_wait(o_empty, (item & 1) ^ 1, p.status, abort_flag))) break;
                    fence_proxy_async_smem();
                    tc_fence_after();
                    const uint32_t tile = ring + st * kStage, weights = p_addr + (it & 1) * kPlan.p_bytes;
#pragma unroll
                    for (int m = 0; m < 4; ++m)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint64_t a = sdesc_mn_sw128(tile + m * kChunk + 4096 * k, kChunk);
                            const uint32_t more = (t != w.t0 || k != 0) ? 1u : 0u;
                            if (kWide) {
#pragma unroll
                                for (int i = 0; i < 3; ++i)
                                    mma_fp8(tmem + m * kOCols, a, sdesc_mn_sw64(weights + 4096 * i + 2048 * k), kIdO, i ? 1u : more);
                            } else {
                                mma_fp8(tmem + m * kOCols, a,
                                        N == 16 ? sdesc_mn_sw64(weights + 2048 * k) : sdesc_mn_sw128(weights + 4096 * k, kChunk),
                                        kIdO, more);
                            }
                        }
                    mma_commit(empty + st);
                    mma_commit(pv_done + (it & 1));
                    if (++st == kStages) st = 0;
                }
                ++item;
            }
            mma_commit(drain + 1);
            mbar_wait(drain + 1, 0, p.status, nullptr);
        }
    } else if (warp >= 4) {
        // ---- softmax and epilogue ----
        const int sw = warp & 3, half = warp >> 3;      // lane quadrant; which half (one: all) of the heads
        const int tid = 128 * half + (threadIdx.x & 127);
        const uint32_t lanes = static_cast<uint32_t>(32 * sw) << 16;
        const int key = 16 * sw + (lane & 15);
        const int hw = half * (N / kHalves), hb = hw + (lane >> 4) * kH;     // this warp's and this thread's first head
        uint32_t it = 0, item = 0, st = 0, ph = 0;
        bool ok = true;
        while (ok && walk.next(p, w)) {
            // maximum and this thread's share of the sum of head hb + i; the
            // largest scale so far, as a power of two, and what brings it to kTop
            float mx[kH], sum[kH], top = 0x1p-100f, up = kTop * 0x1p100f;
#pragma unroll
            for (int i = 0; i < kH; ++i) {
                mx[i] = kNone;
                sum[i] = 0.0f;
            }
            const float* factor = factors + item % kFactors * N + hb;
            for (int t = w.t0; t < w.t1; ++t, ++it) {
                ok = ok && mbar_wait(s_full + (it & 1), (it >> 1) & 1, p.status, abort_flag);
                tc_fence_after();
                uint32_t raw[kH], low[kH];
                tmem_ld_halves(tmem + lanes + kSCol + (it & 1) * 2 * N + hw, raw);
                tmem_ld_halves(tmem + lanes + kSCol + (it & 1) * 2 * N + N + hw, low);
                // (long complete; it is what makes the copied scales visible here)
                ok = ok && mbar_wait(full + st, ph, p.status, abort_flag);
                const bool valid = (masks[4 * st + sw] >> (lane & 15)) & 1;
                const float scale = scales[st * kKeys + key];
                // x: log2 of the weight, before the maximum goes off
                float x[kH];
#pragma unroll
                for (int i = 0; i < kH; i += 4) *reinterpret_cast<float4*>(x + i) = *reinterpret_cast<const float4*>(factor + i);
                tmem_wait_halves(raw);
                tmem_wait_halves(low);
                tc_fence_before();
                mbar_arrive(s_empty + (it & 1));
                bool grow = !ok || (valid && scale > top);
#pragma unroll
                for (int i = 0; i < kH; ++i) {
                    x[i] = valid ? fmaf(__uint_as_float(low[i]), 0.0625f, __uint_as_float(raw[i])) * scale * x[i] : -INFINITY;
                    grow |= x[i] - mx[i] > kGrow;
                }
                if (named_any<1, kSoftThreads>(grow)) {
                    // a wait that ran out in any thread ends the loop in all
                    if (named_any<1, kSoftThreads>(!ok)) { ok = false; break; }
                    // new maxima: over this warp's 16 keys, then over the four warps
                    float v[kH];
#pragma unroll
                    for (int i = 0; i < kH; ++i) v[i] = x[i];
                    const float most = over_keys(v, [](float a, float b) { return fmaxf(a, b); });
                    if ((lane & 15) < kH) stat[sw * N + hb + (lane & 15)] = most;
                    float s = valid ? scale : 0.0f;
                    for (int d = 8; d > 0; d >>= 1) s = fmaxf(s, __shfl_xor_sync(~0u, s, d));
                    if (half == 0 && lane == 0) stat[5 * N + sw] = s;
                    named_sync<1, kSoftThreads>();
                    s = fmaxf(fmaxf(stat[5 * N], stat[5 * N + 1]), fmaxf(stat[5 * N + 2], stat[5 * N + 3]));
                    // the power of two at or above it
                    s = __uint_as_float((__float_as_uint(fmaxf(s, top)) + 0x7FFFFFu) & 0x7F800000u);
                    const float fall = __fdividef(top, s);
                    top = s;
                    up = __fdividef(kTop, s);
#pragma unroll
                    for (int i = 0; i < kH; ++i) {
                        const int h = hb + i;
                        const float m = fmaxf(fmaxf(fmaxf(stat[h], stat[N + h]), fmaxf(stat[2 * N + h], stat[3 * N + h])), mx[i]);
                        const float f = exp2_fast(mx[i] - m);
                        mx[i] = m;
                        sum[i] *= f;
                        if (sw == 0 && (lane & 15) == 0) stat[4 * N + h] = f * fall;
                    }
                    named_sync<1, kSoftThreads>();
                    if (t != w.t0) {
                        // the accumulators' columns (heads) times their factors,
                        // half of the dimensions each
                        ok = mbar_wait(pv_done + ((it - 1) & 1), ((it - 1) >> 1) & 1, p.status, abort_flag);
                        tc_fence_after();
                        for (int c = kGroupsM * kOCols * half; c < kGroupsM * kOCols * (half + 1); c += 16) {
                            uint32_t v[16];
                            tmem_ld16_nowait(tmem + lanes + c, v);
                            tmem_wait_ld16(v);
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                v[j] = __float_as_uint(__uint_as_float(v[j]) * stat[4 * N + ((c + j) & (N - 1))]);
                            tmem_st16(tmem + lanes + c, v);
                        }
                        tmem_wait_st();
                    }
                }
                // weights, times the scale, as three e5m2
                const float by = scale * up;
                uint32_t part[3][kH / 4];
#pragma unroll
                for (int i = 0; i < kH; i += 4) {
                    float e[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        e[k] = exp2_fast(x[i + k] - mx[i + k]);
                        sum[i + k] += e[k];
                        e[k] = valid ? e[k] * by : 0.0f;
                    }
                    uint32_t r[2] = {f16x2(e[0], e[1]), f16x2(e[2], e[3])};
#pragma unroll
                    for (int k = 0; k < 3; ++k) {
                        const uint32_t a = to_e5m2(r[0]), b = to_e5m2(r[1]);
                        part[k][i / 4] = __byte_perm(a, b, 0x7531);
                        r[0] = sub_f16x2(r[0], a & kUpper);
                        r[1] = sub_f16x2(r[1], b & kUpper);
                    }
                }
                // the weight tile before last was read
                if (it > 1) ok = mbar_wait(pv_done + (it & 1), ((it >> 1) & 1) ^ 1, p.status, abort_flag) && ok;
                uint8_t* pt = smem + kPlan.p_off + (it & 1) * kPlan.p_bytes;
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    // rows are keys: of N bytes in each of three tiles, of 3 N bytes in one
                    if constexpr (N == 64) {
                        *reinterpret_cast<uint4*>(pt + 4096 * k + key * 64 + (((hb >> 4) ^ ((key >> 1) & 3)) << 4)) =
                            *reinterpret_cast<const uint4*>(part[k]);
                    } else if constexpr (N == 32) {
                        *reinterpret_cast<uint4*>(pt + key * 128 + (((2 * k + (hb >> 4)) ^ (key & 7)) << 4)) =
                            *reinterpret_cast<const uint4*>(part[k]);
                    } else {
                        *reinterpret_cast<uint2*>(pt + key * 64 + ((k ^ ((key >> 1) & 3)) << 4) + hb) =
                            *reinterpret_cast<const uint2*>(part[k]);
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(p_full + (it & 1));
                if (++st == kStages) st = 0, ph ^= 1;
            }
            // A wait may have run out in some threads alone.  None of them leaves
            // before the vote below, whose barrier counts every thread.
            // sums over the warp's keys, then over the four warps
            ok = ok && mbar_wait(pv_done + ((it - 1) & 1), ((it - 1) >> 1) & 1, p.status, abort_flag);
            tc_fence_after();
            {
                const float all = over_keys(sum, [](float a, float b) { return a + b; });
                if ((lane & 15) < kH) stat[sw * N + hb + (lane & 15)] = all;
                if (sw == 0 && (lane & 15) == 0) {
#pragma unroll
                    for (int i = 0; i < kH; ++i) stat[4 * N + hb + i] = mx[i];
                }
            }
            if (named_any<1, kSoftThreads>(!ok)) { ok = false; break; }
            const float unit = top * (1.0f / kTop);      // of the accumulators
            if constexpr (kCl > 1) {
                // this CTA's share to its own shared memory (everything in front of the
                // statistics is consumed): statistics, then the accumulators [head][512]
                float2 ml = make_float2(0.0f, 0.0f);
                if (tid < N) ml = make_float2(stat[4 * N + tid], stat[tid] + stat[N + tid] + stat[2 * N + tid] + stat[3 * N + tid]);
                named_sync<1, kSoftThreads>();
                if (tid < N) reinterpret_cast<float2*>(stat)[tid] = ml;
                float* share = reinterpret_cast<float*>(smem) + 128 * kGroupsM * half + 32 * sw + lane;
#pragma unroll 1
                for (int hc = 0; hc < N; hc += 16) {
#pragma unroll 1
                    for (int m = 0; m < kGroupsM; ++m) {
                        float o[16];
#pragma unroll
                        for (int k = 0; k < kOCols / N; ++k) {
                            float v[16];
                            tmem_ld16(tmem + lanes + (kGroupsM * half + m) * kOCols + k * N + hc, v);
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] = k ? o[j] + v[j] : v[j];
                        }
#pragma unroll
                        for (int j = 0; j < 16; ++j) share[(hc + j) * IDX_LATENT_DIM + 128 * m] = o[j] * unit;
                    }
                }
                break;      // a cluster's CTA has one piece
            }
            const int h0 = w.hg * 64;
            if (tid < N) {
                const float l = stat[tid] + stat[N + tid] + stat[2 * N + tid] + stat[3 * N + tid];
                const float m = stat[4 * N + tid];
                if (w.slot >= 0)
                    p.part_ml[static_cast<int64_t>(w.slot) * N + tid] = make_float2(m, l);
                else if (p.lse != nullptr && h0 + tid < p.heads)
                    p.lse[w.row * p.heads + h0 + tid] =
                        l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
                // factor of the head's result (partial sums keep their weights)
                stat[4 * N + tid] = w.slot >= 0 ? unit : l == 0.0f ? 0.0f : __fdiv_rn(unit, l);
            }
            named_sync<1, kSoftThreads>();
            // lane = latent dimension, column = head: 16 heads at a time
#pragma unroll 1
            for (int hc = 0; hc < N; hc += 16) {
                float f[16];
#pragma unroll
                for (int j = 0; j < 16; j += 4)
                    *reinterpret_cast<float4*>(f + j) = *reinterpret_cast<const float4*>(stat + 4 * N + hc + j);
                const int d0 = 128 * kGroupsM * half + 32 * sw + lane;
                // neighbouring lanes swap so that each stores two dimensions of one head
                const bool odd = lane & 1;
                const int left = p.heads - h0 - hc - odd;      // heads from this lane's first one on
                __nv_bfloat16* dst = p.out + (w.row * p.heads + h0 + hc + odd) * IDX_LATENT_DIM + (d0 & ~1);
                float* part = p.part_o + (static_cast<int64_t>(w.slot) * N + hc) * IDX_LATENT_DIM + d0;
#pragma unroll 1
                for (int m = 0; m < kGroupsM; ++m) {
                    float o[16];
#pragma unroll
                    for (int k = 0; k < kOCols / N; ++k) {
                        float v[16];
                        tmem_ld16(tmem + lanes + (kGroupsM * half + m) * kOCols + k * N + hc, v);
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] = k ? o[j] + v[j] : v[j];
                    }
                    if (w.slot >= 0) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) part[j * IDX_LATENT_DIM + 128 * m] = o[j] * f[j];
                        continue;
                    }
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        const float a = o[j] * f[j], b = o[j + 1] * f[j + 1];
                        const float c = __shfl_xor_sync(~0u, odd ? a : b, 1);
                        const uint32_t two = odd ? bf16x2(c, b) : bf16x2(a, c);
                        if (j < left) *reinterpret_cast<uint32_t*>(dst + j * IDX_LATENT_DIM + 128 * m) = two;
                    }
                }
            }
            tc_fence_before();
            mbar_arrive(o_empty);
            named_sync<1, kSoftThreads>();   // the statistics' memory is reused
            ++item;
        }
        // a share without tiles
        if (kCl > 1 && it == 0 && tid < N) reinterpret_cast<float2*>(stat)[tid] = make_float2(kNone, 0.0f);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
    if constexpr (kCl > 1) {
        // ---- join: N / kCl heads a CTA, every thread ----
        constexpr int kShare = N / kCl;
        const int rank = static_cast<int>(cluster_rank());
        cluster_arrive();
        cluster_wait();
        const int64_t row = sh_run[2];
        const int h0 = static_cast<int>(sh_run[3]) * 64;
        for (int i = threadIdx.x; i < kShare * (IDX_LATENT_DIM / 4); i += threads_of(N)) {
            const int h = rank * kShare + i / (IDX_LATENT_DIM / 4), d = 4 * (i % (IDX_LATENT_DIM / 4));
            if (h0 + h >= p.heads) continue;
            float2 ml[kCl];
            float4 v[kCl];
            float m = kNone, l = 0.0f;
#pragma unroll
            for (int r = 0; r < kCl; ++r) {
                const uint2 b = dsmem_ld_v2(dsmem_addr(stat + 2 * h, r));
                ml[r] = make_float2(__uint_as_float(b.x), __uint_as_float(b.y));
                v[r] = dsmem_ld_f4(dsmem_addr(smem + (h * IDX_LATENT_DIM + d) * 4, r));
                if (ml[r].y != 0.0f) m = fmaxf(m, ml[r].x);
            }
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int r = 0; r < kCl; ++r) {
                if (ml[r].y == 0.0f) continue;      // nothing there: neither are its sums
                const float f = exp2_fast(ml[r].x - m);
                l += ml[r].y * f;
                o.x += v[r].x * f;
                o.y += v[r].y * f;
                o.z += v[r].z * f;
                o.w += v[r].w * f;
            }
            const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
            const int64_t at = row * p.heads + h0 + h;
            *reinterpret_cast<uint2*>(p.out + at * IDX_LATENT_DIM + d) =
                make_uint2(bf16x2(o.x * inv, o.y * inv), bf16x2(o.z * inv, o.w * inv));
            if (d == 0 && p.lse != nullptr) p.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
        }
        // nobody leaves while another still reads its share
        cluster_arrive();
        cluster_wait();
    }
}

// What joining cut rows costs, in tiles.
constexpr int kJoinTiles = 14;

Shape shape_of(int64_t rows, int heads, int64_t max_keys, bool paged) {
    Shape s{};
    s.N = width_of(heads);
    s.hgs = (heads + 63) / 64;
    s.cluster = 1;
    const int64_t g = kMaxCtas;
    const int64_t items = rows * s.hgs, nt = max_keys > 0 ? (max_keys + kKeys - 1) / kKeys : 1;
    int64_t best = (items + g - 1) / g * nt;
    s.ctas = static_cast<int>(items < g ? items : g);
    for (int c = 2; c <= 8; c *= 2) {
        const int64_t cost = (nt + c - 1) / c + 1;
        if (items * c <= (c == 8 ? 64 : c == 4 ? 128 : g) && c <= nt && cost < best && !(paged && nt > 16)) {
            best = cost;
            s.split = 2;
            s.cluster = c;
            s.ctas = static_cast<int>(items) * c;
        }
    }
    const int64_t cut = (items * nt + g - 1) / g + kJoinTiles;
    if (cut < best) {
        s.split = 1;
        s.cluster = 1;
        const int64_t n = (items * nt + kMinRun - 1) / kMinRun;
        s.ctas = static_cast<int>(n < g ? n : g);
    }
    return s;
}

template <int N, int kCl>
cudaError_t launch_n(const QParams& p, int ctas, cudaStream_t st) {
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = set_smem_once(qattend_kernel<N, kCl>, qplan_of(N).total, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    cfg.blockDim = dim3(threads_of(N), 1, 1);
    cfg.dynamicSmemBytes = qplan_of(N).total;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kCl;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = kCl > 1 ? 2 : 1;
    kt_mark(st);
    e = cudaLaunchKernelEx(&cfg, qattend_kernel<N, kCl>, p);
    kt_mark(st);
    if (e != cudaSuccess || p.split != 1) return e;
    return launch_join(p, N, ctas, st);
}

template <int N>
cudaError_t launch_cl(const QParams& p, const Shape& s, cudaStream_t st) {
    switch (s.cluster) {
        case 2: return launch_n<N, 2>(p, s.ctas, st);
        case 4: return launch_n<N, 4>(p, s.ctas, st);
        case 8: return launch_n<N, 8>(p, s.ctas, st);
        default: return launch_n<N, 1>(p, s.ctas, st);
    }
}

}  // namespace

// Partial sums and statistics of two pieces a CTA.
size_t qattend_ws_need(int64_t rows, int heads, int64_t max_keys, bool paged) {
    const Shape s = shape_of(rows, heads, max_keys, paged);
    if (s.split != 1) return 256;
    return 256 + align_up(static_cast<size_t>(2 * s.ctas) * s.N * (IDX_LATENT_DIM + 2) * 4, 256);
}

cudaError_t launch_qattend(const AttendArgs& a, int64_t block_bytes, cudaStream_t st) {
    const Shape s = shape_of(a.rows, a.heads, a.max_keys, a.block_table != nullptr);
    QParams p{};
    p.slots = a.slots; p.slots_stride = a.slots_stride;
    p.block_table = a.block_table; p.seq_lens = a.seq_lens; p.mbps = a.mbps; p.block_size = a.block_size;
    p.pool = static_cast<const uint8_t*>(a.pool);
    p.rows = a.rows; p.num_slots = a.num_slots; p.heads = a.heads; p.hgs = s.hgs; p.max_keys = a.max_keys;
    p.split = s.split;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.out = static_cast<__nv_bfloat16*>(a.out); p.lse = a.lse; p.status = a.status;
    p.part_o = static_cast<float*>(a.ws);
    p.part_ml = reinterpret_cast<float2*>(p.part_o + static_cast<size_t>(2) * s.ctas * s.N * IDX_LATENT_DIM);
    p.ql = static_cast<const uint16_t*>(a.ql); p.qp = static_cast<const uint16_t*>(a.qp);
    p.ql_row = a.ql_row; p.ql_head = a.ql_head; p.qp_row = a.qp_row; p.qp_head = a.qp_head;
    p.block_bytes = block_bytes;
    if (s.N == 16) return launch_cl<16>(p, s, st);
    if (s.N == 32) return launch_cl<32>(p, s, st);
    return launch_cl<64>(p, s, st);
}

}  // namespace dsaidx
