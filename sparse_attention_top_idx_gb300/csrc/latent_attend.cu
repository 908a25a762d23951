// latent_attend.cu -- absorbed latent attention over selected slots or a paged
// context.
//
// Mathematics, for one row (a query of up to 64 heads) and tiles of 64 keys
// with records [c | p]:
//   S^T = K Q^T           [64 keys, heads],  K = [c | p], 36 steps of 16
//   P   = 2^(S scale log2(e) - m)            per head, masked keys 0
//   O^T = c^T P^T         [512, heads]       accumulated over the tiles
// Keys are the rows of the score product and latent dimensions those of the
// value product, so a call with few heads (16, 32) issues narrow products
// instead of padding its heads to 64 or 128 rows, and the tile that the rows'
// gather leaves in shared memory is the operand of both products: K-major for
// the scores, MN-major for the values.
//
// One persistent CTA an SM, warp-specialised:
//   warp 0     one lane issues the score products, up to two tiles ahead of
//              the softmax
//   warp 1     loads a row's queries
//   warp 2     one lane issues the value products.  (One lane for both was the
//              kernel's bound: its polling and 56 issues took 3400 cycles a
//              tile.)
//   warps 4-7, at 64 heads 12-15 too  softmax, half of the heads each, and
//              epilogue, half of the dimensions each
//   warps 8-11 gather records, 16 keys of every tile each, with 16-byte
//              asynchronous copies into a ring of chunk pairs (128 latent
//              dimensions of 64 keys) and one of position chunks; masked keys
//              are filled with zeros.  Every thread reports its copies twice
//              a tile (128 reports a pair took 5 % at 64 heads).  (TMA's row
//              gather took 42 ns for four 128-byte rows, 6.1 us a tile.)
// A chunk pair is freed by the value product that reads it last, so the next
// tile's loads start while this tile's products run.
//
// The running maximum of a head moves only when a score passes it by 2^8
// (weights stay below 256, in fp32 and in bf16 with the same relative error),
// so most tiles need neither a maximum over keys nor a rescaled accumulator:
// one barrier with an OR decides for all heads.  Weights are rounded to bf16
// for the value product (relative 2^-8 at most, as large as the rounding of
// the result); their sums, the statistics and both accumulators are fp32.
//
// Few rows over many keys: the tiles of all rows form one line that is cut
// into equal runs, one a CTA; a row that is cut leaves partial sums (fp32) in
// the workspace, which a second kernel joins in the order of the keys.  Few
// rows over few keys: the CTAs of a cluster share a row's tiles, leave their
// partial sums in shared memory and join each other's, a share of the heads
// each, through it.
//
// Measured: a tile takes 1.26 us at 16 heads (58 bytes a ns and SM, the rate of
// the copies themselves: without products or without reading memory it stays;
// long contexts: 6.6 TB/s, bound by HBM) and 1.40 us at 64 (152 rows of 16,384
// keys each).  4096 rows of 1024 keys, 128 heads: 1.38 ms, 846 TFLOP/s, 1.60 us
// a tile with the rows' beginnings and ends; 1.37 us of it are the steps of the
// products (36 of 64 keys x 64 heads at 24 ns, 16 of 128 dimensions x 64 heads
// at 32 ns, two issuing warps; 10.4 and 20.8 ns at the measured 1912 TFLOP/s).
#include <cuda_bf16.h>

#include <cmath>

#include "internal.h"
#include "latent.h"
#include "latent_map.h"
#include "latent_mma.cuh"

namespace dsaidx {

namespace {

constexpr int kKeys = 64;                  // keys a tile
constexpr int kChunk = kKeys * 128;        // bytes of a chunk: 64 keys x 64 values
constexpr int kPair = 2 * kChunk;
// Softmax warpgroups: two at 64 heads (4096 rows of 1024 keys, 128 heads, 1.43
// ms against 1.53, as a row's epilogue halves); at 16 a second one costs 3 %.
constexpr int halves_of(int N) { return N == 64 ? 2 : 1; }
constexpr int threads_of(int N) { return 256 + 128 * halves_of(N); }
constexpr int kGatherThreads = 128;
constexpr int kMaxCtas = 152;              // one an SM; CTAs of different clusters never wait on one another
constexpr int kMinRun = 2;                 // tiles a CTA, at least, where rows are cut
constexpr float kNone = -3.0e38f;          // maximum of a head without a key so far
constexpr float kGrow = 8.0f;              // log2 by which a score may pass the maximum

// Shared memory: queries, weights, the pair ring, two position chunks, then
// masks, statistics and barriers.
struct Plan {
    int pairs, q_off, p_off, ring_off, pe_off, stat_off, mask_off, bar_off, total;
};
__host__ __device__ constexpr Plan plan_of(int N) {
    Plan p{};
    p.pairs = N == 64 ? 8 : N == 32 ? 10 : 11;   // a tile takes four
    int o = 0;
    p.q_off = o;    o += 9 * N * 128;
    p.p_off = o;    o += kChunk;
    p.ring_off = o; o += p.pairs * kPair;
    p.pe_off = o;   o += 2 * kChunk;
    p.stat_off = o; o += 5 * N * 4;        // four warps' values and one for all
    p.mask_off = o; o += 4 * 8;
    p.bar_off = o;  o += (p.pairs + 24) * 8;
    p.total = o + 1024;
    return p;
}
static_assert(plan_of(64).total <= 232448 && plan_of(32).total <= 232448 && plan_of(16).total <= 232448,
              "fits one SM's shared memory");

struct Params {
    const int64_t* slots;
    int64_t slots_stride;
    const int32_t* block_table;
    const int32_t* seq_lens;
    int64_t rows, num_slots;
    int block_size, mbps, heads, hgs, max_keys;
    int split;                 // 0: whole rows; 1: the tiles of all rows in equal runs; 2: a row's tiles over a cluster
    int ql_swap, qp_swap;      // the map's middle dimension is the row
    const uint8_t* pool;
    float scale_log2;
    __nv_bfloat16* out;
    float* lse;
    int32_t* status;
    float* part_o;             // [2 ctas][N][512]
    float2* part_ml;           // [2 ctas][N]
};

// Visible keys of a row: its length where that is in range, else 0.
__device__ __forceinline__ int row_keys(const Params& p, int64_t row) {
    if (p.block_table == nullptr) return p.max_keys;
    const int n = __ldg(p.seq_lens + row);
    if (n < 0 || n > p.max_keys || n > static_cast<int64_t>(p.mbps) * p.block_size) return 0;
    return n;
}
// Tiles of a row; one for an empty row, which still writes its result.
__device__ __forceinline__ int tiles_of(int keys) { return keys > 0 ? (keys - 1) / kKeys + 1 : 1; }

// Where the run of CTA c of g begins in the line of tt tiles.
__device__ __forceinline__ int64_t run_start(int64_t c, int64_t g, int64_t tt) { return c * tt / g; }

// Row in whose tiles position x of the line lies, and where the row begins
// (both scaled by the head groups); with x < 0 the length of the line.
// Executed by a whole warp; paged contexts only.
__device__ __forceinline__ void find_row(const Params& p, int64_t x, int64_t& row, int64_t& base) {
    const int lane = lane_id();
    int64_t acc = 0;
    for (int64_t r0 = 0; r0 < p.rows; r0 += 32) {
        const int64_t r = r0 + lane;
        int64_t v = r < p.rows ? static_cast<int64_t>(tiles_of(row_keys(p, r))) * p.hgs : 0;
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

// One piece of work: tiles [t0, t1) of a row's head group.
struct Work {
    int64_t row;
    int hg, keys, t0, t1;
    int slot;       // where its partial sums go; -1: it has all tiles, write the result; -2: the cluster joins
};

// The pieces of this CTA, in order; every role walks them by itself.
struct Walk {
    int64_t pos, end;        // split: the run left; whole: item and number of items
    int64_t row, base;       // split, paged: current row and where it begins; cluster: row and head group
    bool first;
    __device__ __forceinline__ Walk(const Params& p, int64_t start, int64_t end_, int64_t row_, int64_t base_)
        : pos(start), end(end_), row(row_), base(base_), first(true) {}
    __device__ __forceinline__ bool next(const Params& p, Work& w) {
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
            w.row = pos / p.hgs;
            w.hg = static_cast<int>(pos - w.row * p.hgs);
            w.keys = row_keys(p, w.row);
            w.t0 = 0;
            w.t1 = tiles_of(w.keys);
            w.slot = -1;
            pos += gridDim.x;
            return true;
        }
        int64_t in;
        int nt;
        if (p.block_table == nullptr) {
            w.keys = p.max_keys;
            nt = tiles_of(w.keys);
            const int64_t item = pos / nt;
            w.row = item / p.hgs;
            w.hg = static_cast<int>(item - w.row * p.hgs);
            in = pos - item * nt;
        } else {
            w.keys = row_keys(p, row);
            nt = tiles_of(w.keys);
            if (pos - base >= static_cast<int64_t>(nt) * p.hgs) {
                base += static_cast<int64_t>(nt) * p.hgs;
                ++row;
                w.keys = row_keys(p, row);
                nt = tiles_of(w.keys);
            }
            w.row = row;
            w.hg = static_cast<int>((pos - base) / nt);
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
__device__ __forceinline__ int64_t key_entry(const Params& p, int64_t row, int keys, int j) {
    if (j >= keys) return -1;
    return p.block_table == nullptr ? __ldg(p.slots + row * p.slots_stride + j)
                                    : static_cast<int64_t>(__ldg(p.block_table + row * p.mbps + j / p.block_size));
}
// Slot of key j; num_slots where it is masked.
__device__ __forceinline__ int key_slot(const Params& p, int keys, int j, int64_t entry) {
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

template <int N, int kCl>
__global__ void __launch_bounds__(threads_of(N), 1)
    attend_kernel(const __grid_constant__ CUtensorMap ql_map, const __grid_constant__ CUtensorMap qp_map,
                  const Params p) {
    constexpr Plan kPlan = plan_of(N);
    constexpr int kHalves = halves_of(N), kSoftThreads = 128 * kHalves, kGroupsM = 4 / kHalves;
    constexpr int kPairs = kPlan.pairs;
    constexpr int kSPitch = N < 32 ? 32 : N;   // TMEM columns of a score buffer
    constexpr int kSCol = 4 * N;               // first column behind the accumulators
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + kPlan.bar_off);
    uint64_t* pair_empty = bar;
    uint64_t* pe_empty = bar + kPairs;           // [2]
    uint64_t* half_full = pe_empty + 2;          // [2 tiles][2]: position chunk and two pairs, two pairs
    uint64_t* s_full = pe_empty + 6;             // [2]
    uint64_t* s_empty = pe_empty + 8;            // [2]
    uint64_t* p_full = pe_empty + 10;
    uint64_t* pv_done = pe_empty + 11;
    uint64_t* q_full = pe_empty + 12;
    uint64_t* q_empty = pe_empty + 13;
    uint64_t* o_empty = pe_empty + 14;
    uint64_t* drain = pe_empty + 15;             // [2]
    int64_t* sh_run = reinterpret_cast<int64_t*>(pe_empty + 17);   // start, end, row, base
    uint32_t* sh_tmem = reinterpret_cast<uint32_t*>(pe_empty + 21);
    int* sh_abort = reinterpret_cast<int*>(sh_tmem + 1);
    uint16_t* masks = reinterpret_cast<uint16_t*>(smem + kPlan.mask_off);   // [4 tiles][4]: 16 keys each
    float* stat = reinterpret_cast<float*>(smem + kPlan.stat_off);          // [5][N]
    const int warp = warp_id(), lane = lane_id();

    if (warp == 0 && elect_one()) {
        for (int i = 0; i < kPairs; ++i) mbar_init(pair_empty + i, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(pe_empty + i, 1);
            mbar_init(s_full + i, 1);
        }
        for (int i = 0; i < 4; ++i) mbar_init(half_full + i, kGatherThreads + kGatherThreads / 32);
        mbar_init(p_full, kSoftThreads);
        mbar_init(pv_done, 1);
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(o_empty, kSoftThreads);
        mbar_init(drain, 1);
        mbar_init(drain + 1, 1);
        mbar_init(s_empty, kSoftThreads);
        mbar_init(s_empty + 1, kSoftThreads);
        *sh_abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(sh_tmem, 512);
        tmem_relinquish();
    }
    if (warp == 2 && elect_one()) {
        tma_prefetch_desc(&ql_map);
        tma_prefetch_desc(&qp_map);
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
        // ---- gather: 16 keys of every tile ----
        // A copy instruction moves 128 bytes of four keys: lane / 8 is the key
        // among them, lane % 8 the 16-byte piece.
        const int wq = warp - 8, sub = lane >> 3, piece = lane & 7;
        const uint32_t even = wq * 2048 + sub * 128 + ((piece ^ sub) << 4), odd = even ^ 64u;   // keys 4 k + sub by k
        const uint32_t ring = smem_u32(smem + kPlan.ring_off), pe = smem_u32(smem + kPlan.pe_off);
        const int none = static_cast<int>(p.num_slots), j = 16 * wq + (lane & 15);
        uint32_t it = 0, sl = 0, ph = 1;      // tiles, ring slot and the parity that frees it
        bool ok = true;
        while (ok && walk.next(p, w)) {
            if (p.block_table != nullptr && w.keys == 0 && lane == 0 && __ldg(p.seq_lens + w.row) != 0)
                set_status(p.status, IDX_ERR_DEVICE_CHECK);
            int64_t entry = key_entry(p, w.row, w.keys, w.t0 * kKeys + j);
            for (int t = w.t0; t < w.t1; ++t, ++it) {
                const int slot = key_slot(p, w.keys, t * kKeys + j, entry);
                const uint32_t valid = __ballot_sync(~0u, slot != none) & 0xFFFFu;
                const uint8_t* src[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int s = __shfl_sync(~0u, slot, 4 * k + sub);
                    src[k] = p.pool + static_cast<int64_t>(s == none ? 0 : s) * (IDX_LATENT_RECORD * 2) + 16 * piece;
                }
                if (t + 1 < w.t1) entry = key_entry(p, w.row, w.keys, (t + 1) * kKeys + j);
                auto chunk = [&](uint32_t dst, int c) {
                    if (valid == 0xFFFFu) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) copy16(dst + ((k & 1) ? odd : even) + 512 * k, src[k] + 128 * c);
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            copy16_or_zero(dst + ((k & 1) ? odd : even) + 512 * k, src[k] + 128 * c,
                                           (valid >> (4 * k + sub)) & 1 ? 16 : 0);
                    }
                };
                ok = mbar_wait(pe_empty + (it & 1), ((it >> 1) & 1) ^ 1, p.status, abort_flag);
                if (!(ok = __all_sync(~0u, ok))) break;
                if (lane == 0) masks[4 * (it & 3) + wq] = static_cast<uint16_t>(valid);
                chunk(pe + (it & 1) * kChunk, 8);
#pragma unroll 1
                for (int m = 0; m < 4; ++m) {
                    ok = mbar_wait(pair_empty + sl, ph, p.status, abort_flag);
                    if (!(ok = __all_sync(~0u, ok))) break;
                    const uint32_t dst = ring + sl * kPair;
                    chunk(dst, 2 * m);
                    chunk(dst + kChunk, 2 * m + 1);
                    if (m & 1) {
                        // what this thread issued for the half, and the mask
                        uint64_t* full = half_full + 2 * (it & 1) + (m >> 1);
                        copy_arrive(full);
                        if (lane == 0) mbar_arrive(full);
                    }
                    if (++sl == kPairs) sl = 0, ph ^= 1;
                }
                if (!ok) break;
            }
        }
        copy_wait_all();
    } else if (warp == 0) {
        // ---- score products ----
        if (elect_one()) {
            constexpr uint32_t kIdS = idesc_bf16(64, N, false, false);
            const uint32_t q_addr = smem_u32(smem + kPlan.q_off), ring = smem_u32(smem + kPlan.ring_off);
            const uint32_t pe_addr = smem_u32(smem + kPlan.pe_off);
            uint32_t it = 0, item = 0, sl = 0;
            bool ok = true;
            while (ok && walk.next(p, w)) {
                if (!(ok = mbar_wait(q_full, item & 1, p.status, abort_flag))) break;
                for (int t = w.t0; t < w.t1; ++t, ++it) {
                    const uint32_t d = tmem + kSCol + (it & 1) * kSPitch;
                    // the softmax has read the scores before last
                    if (!(ok = mbar_wait(s_empty + (it & 1), ((it >> 1) & 1) ^ 1, p.status, abort_flag))) break;
                    if (!(ok = mbar_wait(half_full + 2 * (it & 1), (it >> 1) & 1, p.status, abort_flag))) break;
                    // the records were copied by other threads: order their
                    // writes before the tensor core's reads
                    fence_proxy_async_smem();
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_bf16(d, sdesc_sw128(pe_addr + (it & 1) * kChunk + 32 * k),
                                 sdesc_sw128(q_addr + 8 * N * 128 + 32 * k), kIdS, k != 0);
                    mma_commit(pe_empty + (it & 1));
#pragma unroll 1
                    for (int m = 0; m < 4; ++m) {
                        if (m == 2) {
                            if (!(ok = mbar_wait(half_full + 2 * (it & 1) + 1, (it >> 1) & 1, p.status, abort_flag))) break;
                            fence_proxy_async_smem();
                            tc_fence_after();
                        }
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            mma_bf16(d, sdesc_sw128(ring + sl * kPair + (k >> 2) * kChunk + 32 * (k & 3)),
                                     sdesc_sw128(q_addr + (2 * m + (k >> 2)) * N * 128 + 32 * (k & 3)), kIdS, 1u);
                        if (++sl == kPairs) sl = 0;
                    }
                    if (!ok) break;
                    mma_commit(s_full + (it & 1));
                    if (t + 1 == w.t1) mma_commit(q_empty);
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
            constexpr uint32_t kIdO = idesc_bf16(128, N, true, true);
            const uint32_t ring = smem_u32(smem + kPlan.ring_off), p_addr = smem_u32(smem + kPlan.p_off);
            uint32_t it = 0, item = 0, sl = 0;
            bool ok = true;
            while (ok && walk.next(p, w)) {
                for (int t = w.t0; t < w.t1; ++t, ++it) {
                    // the weights are there, which the records were before them
                    if (!(ok = mbar_wait(p_full, it & 1, p.status, abort_flag))) break;
                    // the accumulators of the piece before were read
                    if (t == w.t0 && !(ok = mbar_wait(o_empty, (item & 1) ^ 1, p.status, abort_flag))) break;
                    fence_proxy_async_smem();
                    tc_fence_after();
#pragma unroll 1
                    for (int m = 0; m < 4; ++m) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_bf16(tmem + m * N, sdesc_mn_sw128(ring + sl * kPair + 2048 * k, kChunk),
                                     sdesc_mn_sw128(p_addr + 2048 * k, kChunk), kIdO, (t != w.t0 || k != 0) ? 1u : 0u);
                        mma_commit(pair_empty + sl);
                        if (++sl == kPairs) sl = 0;
                    }
                    mma_commit(pv_done);
                }
                ++item;
            }
            mma_commit(drain + 1);
            mbar_wait(drain + 1, 0, p.status, nullptr);
        }
    } else if (warp == 1) {
        // ---- queries ----
        if (elect_one()) {
            uint32_t item = 0;
            bool ok = true;
            while (ok && walk.next(p, w)) {
                ok = mbar_wait(q_empty, (item & 1) ^ 1, p.status, abort_flag);
                if (!ok) break;
                mbar_arrive_expect_tx(q_full, 9 * N * 128);
                const uint32_t q_addr = smem_u32(smem + kPlan.q_off);
                const int h = w.hg * 64, row = static_cast<int>(w.row);
                for (int c = 0; c < 8; ++c)
                    tma_tile_3d(q_addr + c * N * 128, &ql_map, q_full, 64 * c, p.ql_swap ? row : h, p.ql_swap ? h : row);
                tma_tile_3d(q_addr + 8 * N * 128, &qp_map, q_full, 0, p.qp_swap ? row : h, p.qp_swap ? h : row);
                ++item;
            }
            if (item) mbar_wait(q_full, (item - 1) & 1, p.status, nullptr);
        }
    } else if (warp >= 4) {
        // ---- softmax and epilogue ----
        const int sw = warp & 3, half = warp >> 3;      // lane quadrant; which half (one: all) of the heads
        const int tid = 128 * half + (threadIdx.x & 127);
        const uint32_t lanes = static_cast<uint32_t>(32 * sw) << 16;
        const int quad = lane & 3, kr = lane >> 2;      // column pair and key row within the warp's 16
        constexpr int kR = N / 8 / kHalves;             // this half's column groups of 8 heads
        constexpr int kGroups = kR < 4 ? 1 : kR / 4;    // loads of 32 columns
        const int hb = half * (N / kHalves);            // and its first head
        uint32_t it = 0;
        bool ok = true;
        while (ok && walk.next(p, w)) {
            // head hb + 8 r + 2 quad + e: maximum and this thread's share of the sum
            float mx[kR][2], sum[kR][2];
#pragma unroll
            for (int r = 0; r < kR; ++r) {
                mx[r][0] = mx[r][1] = kNone;
                sum[r][0] = sum[r][1] = 0.0f;
            }
            for (int t = w.t0; t < w.t1; ++t, ++it) {
                ok = ok && mbar_wait(s_full + (it & 1), (it >> 1) & 1, p.status, abort_flag);
                tc_fence_after();
                uint32_t raw[kGroups][16];
#pragma unroll
                for (int g = 0; g < (kGroups); ++g)
                    tmem_ld_16x256b_x4(tmem + lanes + kSCol + (it & 1) * kSPitch + hb + 32 * g, raw[g]);
                const uint32_t mask = masks[4 * (it & 3) + sw];
                const bool va = (mask >> kr) & 1, vb = (mask >> (kr + 8)) & 1;
#pragma unroll
                for (int g = 0; g < (kGroups); ++g) tmem_wait_ld16(raw[g]);
                tc_fence_before();
                mbar_arrive(s_empty + (it & 1));
                // y[r][e]: key kr, y[r][2 + e]: key kr + 8; log2 of the weight
                float y[kR][4];
                bool grow = !ok;
#pragma unroll
                for (int r = 0; r < kR; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float s = __uint_as_float(raw[r / 4][4 * (r % 4) + e]);
                        y[r][e] = (e < 2 ? va : vb) ? fmaf(s, p.scale_log2, -mx[r][e & 1]) : -INFINITY;
                        grow |= y[r][e] > kGrow;
                    }
                if (named_any<1, kSoftThreads>(grow)) {
                    // a wait that ran out in any thread ends the loop in all
                    if (named_any<1, kSoftThreads>(!ok)) { ok = false; break; }
                    // new maxima: over this warp's 16 keys, then over the four warps
#pragma unroll
                    for (int r = 0; r < kR; ++r)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float s0 = __uint_as_float(raw[r / 4][4 * (r % 4) + e]);
                            const float s1 = __uint_as_float(raw[r / 4][4 * (r % 4) + 2 + e]);
                            float v = fmaxf(va ? s0 * p.scale_log2 : kNone, vb ? s1 * p.scale_log2 : kNone);
                            v = fmaxf(v, __shfl_xor_sync(~0u, v, 4));
                            v = fmaxf(v, __shfl_xor_sync(~0u, v, 8));
                            v = fmaxf(v, __shfl_xor_sync(~0u, v, 16));
                            if (kr == 0) stat[sw * N + hb + 8 * r + 2 * quad + e] = v;
                        }
                    named_sync<1, kSoftThreads>();
#pragma unroll
                    for (int r = 0; r < kR; ++r)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int h = hb + 8 * r + 2 * quad + e;
                            float v = fmaxf(fmaxf(stat[h], stat[N + h]), fmaxf(stat[2 * N + h], stat[3 * N + h]));
                            v = fmaxf(v, mx[r][e]);
                            const float f = exp2_fast(mx[r][e] - v);
                            mx[r][e] = v;
                            sum[r][e] *= f;
                            if (sw == 0 && kr == 0) stat[4 * N + h] = f;
                            const float s0 = __uint_as_float(raw[r / 4][4 * (r % 4) + e]);
                            const float s1 = __uint_as_float(raw[r / 4][4 * (r % 4) + 2 + e]);
                            y[r][e] = va ? fmaf(s0, p.scale_log2, -v) : -INFINITY;
                            y[r][2 + e] = vb ? fmaf(s1, p.scale_log2, -v) : -INFINITY;
                        }
                    named_sync<1, kSoftThreads>();
                    if (t != w.t0) {
                        // the accumulators' columns (heads) times their factors,
                        // half of the dimensions each
                        ok = mbar_wait(pv_done, (it - 1) & 1, p.status, abort_flag);
                        tc_fence_after();
                        for (int c = kGroupsM * N * half; c < kGroupsM * N * (half + 1); c += 16) {
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
                uint32_t pk[kR][2];
#pragma unroll
                for (int r = 0; r < kR; ++r) {
                    float e[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) e[k] = exp2_fast(y[r][k]);
                    sum[r][0] += e[0] + e[2];
                    sum[r][1] += e[1] + e[3];
                    pk[r][0] = bf16x2(e[0], e[1]);
                    pk[r][1] = bf16x2(e[2], e[3]);
                }
                // weights: row = key, 64 heads of it contiguous
                if (it > 0) ok = mbar_wait(pv_done, (it - 1) & 1, p.status, abort_flag) && ok;
                const int ka = 16 * sw + kr;
                uint8_t* pa = smem + kPlan.p_off + ka * 128 + 4 * quad;
#pragma unroll
                for (int r = 0; r < kR; ++r) {
                    const uint32_t at = ((half * kR + r) ^ (ka & 7)) << 4;
                    *reinterpret_cast<uint32_t*>(pa + at) = pk[r][0];
                    *reinterpret_cast<uint32_t*>(pa + 1024 + at) = pk[r][1];
                }
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(p_full);
            }
            // A wait may have run out in some threads alone.  None of them leaves
            // before the vote below, whose barrier counts every thread.
            // sums over the warp's keys, then over the four warps
            ok = ok && mbar_wait(pv_done, (it - 1) & 1, p.status, abort_flag);
            tc_fence_after();
#pragma unroll
            for (int r = 0; r < kR; ++r)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float v = sum[r][e];
                    v += __shfl_xor_sync(~0u, v, 4);
                    v += __shfl_xor_sync(~0u, v, 8);
                    v += __shfl_xor_sync(~0u, v, 16);
                    if (kr == 0) stat[sw * N + hb + 8 * r + 2 * quad + e] = v;
                    if (sw == 0 && kr == 0) stat[4 * N + hb + 8 * r + 2 * quad + e] = mx[r][e];
                }
            if (named_any<1, kSoftThreads>(!ok)) { ok = false; break; }
            if constexpr (kCl > 1) {
                // this CTA's share to its own shared memory (the ring's loads
                // are all consumed): statistics, then the accumulators [head][512]
                float2 ml = make_float2(0.0f, 0.0f);
                if (tid < N) ml = make_float2(stat[4 * N + tid], stat[tid] + stat[N + tid] + stat[2 * N + tid] + stat[3 * N + tid]);
                named_sync<1, kSoftThreads>();
                if (tid < N) reinterpret_cast<float2*>(stat)[tid] = ml;
                float* share = reinterpret_cast<float*>(smem + kPlan.ring_off) + 128 * kGroupsM * half + 32 * sw + lane;
#pragma unroll 1
                for (int hc = 0; hc < N; hc += 16) {
                    uint32_t v[kGroupsM][16];
#pragma unroll
                    for (int m = 0; m < kGroupsM; ++m) tmem_ld16_nowait(tmem + lanes + (kGroupsM * half + m) * N + hc, v[m]);
#pragma unroll
                    for (int m = 0; m < kGroupsM; ++m) {
                        tmem_wait_ld16(v[m]);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            share[(hc + j) * IDX_LATENT_DIM + 128 * m] = __uint_as_float(v[m][j]);
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
                // factor of the head's result (partial sums stay as they are)
                stat[4 * N + tid] = w.slot >= 0 ? 1.0f : l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
            }
            named_sync<1, kSoftThreads>();
            // lane = latent dimension, column = head: 16 heads at a time, this
            // half's groups of 128 dimensions in flight together
#pragma unroll 1
            for (int hc = 0; hc < N; hc += 16) {
                uint32_t v[kGroupsM][16];
#pragma unroll
                for (int m = 0; m < kGroupsM; ++m) tmem_ld16_nowait(tmem + lanes + (kGroupsM * half + m) * N + hc, v[m]);
                const int d0 = 128 * kGroupsM * half + 32 * sw + lane;
                if (w.slot >= 0) {
                    float* dst = p.part_o + (static_cast<int64_t>(w.slot) * N + hc) * IDX_LATENT_DIM + d0;
#pragma unroll
                    for (int m = 0; m < kGroupsM; ++m) {
                        tmem_wait_ld16(v[m]);
#pragma unroll
                        for (int j = 0; j < 16; ++j) dst[j * IDX_LATENT_DIM + 128 * m] = __uint_as_float(v[m][j]);
                    }
                    continue;
                }
                float f[16];
#pragma unroll
                for (int j = 0; j < 16; j += 4)
                    *reinterpret_cast<float4*>(f + j) = *reinterpret_cast<const float4*>(stat + 4 * N + hc + j);
                // neighbouring lanes swap so that each stores two dimensions of one head
                const bool odd = lane & 1;
                const int left = p.heads - h0 - hc - odd;      // heads from this lane's first one on
                __nv_bfloat16* dst = p.out + (w.row * p.heads + h0 + hc + odd) * IDX_LATENT_DIM + (d0 & ~1);
#pragma unroll
                for (int m = 0; m < kGroupsM; ++m) {
                    tmem_wait_ld16(v[m]);
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        const float a = __uint_as_float(v[m][j]) * f[j], b = __uint_as_float(v[m][j + 1]) * f[j + 1];
                        const float o = __shfl_xor_sync(~0u, odd ? a : b, 1);
                        const uint32_t two = odd ? bf16x2(o, b) : bf16x2(a, o);
                        if (j < left) *reinterpret_cast<uint32_t*>(dst + j * IDX_LATENT_DIM + 128 * m) = two;
                    }
                }
            }
            tc_fence_before();
            mbar_arrive(o_empty);
            named_sync<1, kSoftThreads>();   // the statistics' memory is reused
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
                v[r] = dsmem_ld_f4(dsmem_addr(smem + kPlan.ring_off + (h * IDX_LATENT_DIM + d) * 4, r));
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

// Joins the partial sums of the rows that were cut.  kW warps take the pieces
// of a (row, head) in turn, four of them in flight, lanes over the latent
// dimensions; the warps' sums are added in order.  A CTA has eight warps.
constexpr int kJoinWarps = 8;

template <int kW>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const Params p, int N, int ctas) {
    __shared__ float acc[kW > 1 ? kJoinWarps : 1][IDX_LATENT_DIM];
    __shared__ float factor[kJoinWarps][kMaxCtas];     // of each piece, 0 where there is nothing
    __shared__ int from[kJoinWarps][kMaxCtas];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t row = blockIdx.x;
    const int warp = warp_id(), lane = lane_id(), wh = warp % kW;
    const int head = blockIdx.y * (kJoinWarps / kW) + warp / kW, hg = head / 64, h = head % 64;
    const bool live = head < p.heads;
    int64_t a, tt;
    const int nt = tiles_of(row_keys(p, row));
    if (p.block_table == nullptr) {
        tt = p.rows * p.hgs * nt;
        a = row * p.hgs * nt;
    } else {
        int64_t before = 0, all = 0;
        for (int64_t r = lane; r < p.rows; r += 32) {
            const int64_t t = static_cast<int64_t>(tiles_of(row_keys(p, r))) * p.hgs;
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
            if (start == run_start(c0 + k + 1, ctas, tt)) continue;
            from[warp][k] = static_cast<int>(2 * (c0 + k) + (start < a ? 1 : 0)) * N + h;
            ml[r] = p.part_ml[from[warp][k]];
            if (ml[r].y != 0.0f) m = fmaxf(m, ml[r].x);
        }
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
            float4 v[4][4];
            float f[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int k = k0 + u * kW;
                f[u] = k < pieces ? factor[warp][k] : 0.0f;
                if (f[u] == 0.0f) continue;
                const float4* src = reinterpret_cast<const float4*>(p.part_o + static_cast<int64_t>(from[warp][k]) * IDX_LATENT_DIM);
#pragma unroll
                for (int q = 0; q < 4; ++q) v[u][q] = __ldg(src + 32 * q + lane);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (f[u] == 0.0f) continue;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    o[q].x += v[u][q].x * f[u];
                    o[q].y += v[u][q].y * f[u];
                    o[q].z += v[u][q].z * f[u];
                    o[q].w += v[u][q].w * f[u];
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

// Heads of one score product.
int width_of(int heads) { return heads <= 16 ? 16 : heads <= 32 ? 32 : 64; }

// What joining cut rows costs, in tiles (measured, see shape_of).
int join_tiles(int N) { return N == 64 ? 12 : 9; }

// How the rows are spread over CTAs.
struct Shape {
    int N, hgs, split, ctas, cluster;
};
Shape shape_of(int64_t rows, int heads, int64_t max_keys, bool paged) {
    Shape s{};
    s.N = width_of(heads);
    s.hgs = (heads + 63) / 64;
    s.cluster = 1;
    const int64_t g = kMaxCtas;
    const int64_t items = rows * s.hgs, nt = max_keys > 0 ? (max_keys + kKeys - 1) / kKeys : 1;
    // Tiles one CTA passes, and what joining costs in tiles.  Whole rows:
    // ceil(items / g) rounds of nt.  Clusters of c, while all fit at once (of
    // eight: 64 CTAs; 16 rows of 8 tiles took 25.8 us in eights, 13.7 in fours,
    // 18.5 whole): 1 tile; 64 rows of 32 tiles, 64 heads, 35 us in pairs, 45
    // cut, 54 whole.  Cut: storing and joining partial sums in memory costs
    // about 9 tiles (12 of 64 heads); 200 rows of 16 tiles, 16 heads, 39 us cut
    // and 46 whole, 64 heads 82 and 60.  A paged batch is ragged, which the cut
    // evens out (32 x 4500 / 10000, 16 heads: 55 us, in fours 66), so long
    // contexts take no clusters.
    const int64_t join = join_tiles(s.N);
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
    const int64_t cut = (items * nt + g - 1) / g + join;
    if (cut < best) {
        s.split = 1;
        s.cluster = 1;
        const int64_t n = (items * nt + kMinRun - 1) / kMinRun;
        s.ctas = static_cast<int>(n < g ? n : g);
    }
    return s;
}

template <int N, int kCl>
cudaError_t launch_n(const Params& p, const CUtensorMap& ql, const CUtensorMap& qp, int ctas, cudaStream_t st) {
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = set_smem_once(attend_kernel<N, kCl>, plan_of(N).total, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    cfg.blockDim = dim3(threads_of(N), 1, 1);
    cfg.dynamicSmemBytes = plan_of(N).total;
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
    e = cudaLaunchKernelEx(&cfg, attend_kernel<N, kCl>, ql, qp, p);
    kt_mark(st);
    if (e != cudaSuccess || p.split != 1) return e;
    cfg.numAttrs = 1;
    // warps a (row, head): eight where rows have many pieces, else as many as
    // there is parallelism for.  Measured: 9 rows to 75 pieces, 16 heads, whole
    // call 403 us with one warp, 369 with eight; 32 rows of 3.4 pieces, 128
    // heads, 46 us with one, 57 with four, 74 with eight; 32 rows of 4.8
    // pieces, 16 heads, 58.6, 55.1 and 58.0 us.
    const int warps = ctas > 6 * p.rows * p.hgs ? 8 : p.rows * p.heads <= 1024 ? 4 : 1;
    cfg.gridDim = dim3(static_cast<unsigned>(p.rows), static_cast<unsigned>((p.heads * warps + kJoinWarps - 1) / kJoinWarps), 1);
    cfg.blockDim = dim3(32 * kJoinWarps, 1, 1);
    cfg.dynamicSmemBytes = 0;
    kt_mark(st);
    e = cudaLaunchKernelEx(&cfg, warps == 8 ? join_kernel<8> : warps == 4 ? join_kernel<4> : join_kernel<1>, p, N, ctas);
    kt_mark(st);
    return e;
}

template <int N>
cudaError_t launch_cl(const Params& p, const CUtensorMap& ql, const CUtensorMap& qp, const Shape& s, cudaStream_t st) {
    switch (s.cluster) {
        case 2: return launch_n<N, 2>(p, ql, qp, s.ctas, st);
        case 4: return launch_n<N, 4>(p, ql, qp, s.ctas, st);
        case 8: return launch_n<N, 8>(p, ql, qp, s.ctas, st);
        default: return launch_n<N, 1>(p, ql, qp, s.ctas, st);
    }
}

}  // namespace

// What the call itself uses: partial sums and statistics of two pieces a CTA.
static size_t ws_of(int64_t ctas, int N) {
    return 256 + align_up(static_cast<size_t>(2 * ctas) * N * (IDX_LATENT_DIM + 2) * 4, 256);
}

size_t attend_ws_need(int64_t rows, int heads, int64_t max_keys, bool paged) {
    const Shape s = shape_of(rows, heads, max_keys, paged);
    return s.split == 1 ? ws_of(s.ctas, s.N) : 256;
}

// Rows are cut for some sizes and not for others, so that a call may need more
// than a larger one.  What is asked for covers every call of no more rows,
// heads and keys: rows of nt tiles are cut only where ceil(items nt / g) + join
// is below ceil(items / g) nt, which takes nt > join + 1, and the CTAs of a cut
// call grow with items nt.
size_t attend_ws_bytes(int64_t rows, int heads, int64_t max_keys) {
    const int64_t items = rows * ((heads + 63) / 64), nt = max_keys > 0 ? (max_keys + kKeys - 1) / kKeys : 1;
    if (nt <= join_tiles(16) + 1) return 256;      // the smallest of the widths
    const int64_t n = (items * nt + kMinRun - 1) / kMinRun;
    return ws_of(n < kMaxCtas ? n : kMaxCtas, width_of(heads));
}

cudaError_t launch_attend(const AttendArgs& a, cudaStream_t st) {
    EncodeTiledFn enc = encode_tiled_fn();
    if (!enc) return cudaErrorNotSupported;
    const Shape s = shape_of(a.rows, a.heads, a.max_keys, a.block_table != nullptr);
    Params p{};
    p.slots = a.slots; p.slots_stride = a.slots_stride;
    p.block_table = a.block_table; p.seq_lens = a.seq_lens; p.mbps = a.mbps; p.block_size = a.block_size;
    p.pool = static_cast<const uint8_t*>(a.pool);
    p.rows = a.rows; p.num_slots = a.num_slots; p.heads = a.heads; p.hgs = s.hgs; p.max_keys = a.max_keys;
    p.split = s.split;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.out = static_cast<__nv_bfloat16*>(a.out); p.lse = a.lse; p.status = a.status;
    p.part_o = static_cast<float*>(a.ws);
    p.part_ml = reinterpret_cast<float2*>(p.part_o + static_cast<size_t>(2) * s.ctas * s.N * IDX_LATENT_DIM);
    CUtensorMap ql, qp;
    if (!head_map(&ql, enc, a.ql, IDX_LATENT_DIM, a.ql_row, a.ql_head, a.rows, a.heads, s.N, 1, &p.ql_swap) ||
        !head_map(&qp, enc, a.qp, IDX_LATENT_PE_DIM, a.qp_row, a.qp_head, a.rows, a.heads, s.N, 1, &p.qp_swap))
        return cudaErrorInvalidValue;
    if (s.N == 16) return launch_cl<16>(p, ql, qp, s, st);
    if (s.N == 32) return launch_cl<32>(p, ql, qp, s, st);
    return launch_cl<64>(p, ql, qp, s, st);
}

}  // namespace dsaidx
