// latent_expanded.cu -- expanded causal attention of packed prompts.
//
// Mathematics, for 128 queries of one head and tiles of 128 keys:
//   S = Qn Kn^T + Qp Kp^T   [128 queries, 128 keys]    12 steps of 16
//   P = 2^(S scale log2(e) - m)                         row statistics in fp32
//   O = O + P V             [128 queries, 128]          8 steps of 16
// One CTA takes 256 queries of a head as two such tiles that share every key
// tile.  While one tile is in softmax, the tensor cores run the other's
// products:  PV0(i) QK0(i + 1) PV1(i) QK1(i + 1) ...
//   warp 0      one lane issues every MMA
//   warp 1      one lane loads queries, keys and values by TMA into a ring of
//               eight 16 KB units: three of a tile's keys (128 keys x 64
//               values), two of its values (64 keys x 128), in the order of
//               their use.  Keys i + 1 take the units of values i - 1 (and one
//               of keys i - 1, which are done with before those), values i + 1
//               those of keys i, so two barriers order all reuse
//   warp 2      zeroes the values behind a sequence's end in its last tile
//               (weights there are 0, but 0 * inf is NaN)
//   warps 4-7 and 8-11   softmax of the two tiles, one query a thread
// TMEM: S0 S1 O0 O1, 128 columns each; the weights (bf16) take the place of
// the scores they came from and are the A operand of the value product: 38 ns
// a step against 55 ns from shared memory.
//
// A row's maximum moves only when a score passes it by 2^8 (weights stay
// below 256 in fp32, and bf16 rounds them with the same relative error), so
// that most tiles take one pass over the scores and leave the accumulator
// alone.  Weights are rounded to bf16 for the value product (relative 2^-8 at
// most, as large as the rounding of the result); their sums are taken before
// that.
//
// Measured: 8192 queries on 22,000 keys, 16 heads, 1.05 to 1.06 ms, 1410 to 1430
// TFLOP/s, bound by the tensor cores.  Every wait and commit of the issuing lane
// counts (all on the box where this kernel took 1.02 ms): with a barrier a unit
// (twelve waits a key tile instead of four) 1.15 ms; with a second issuing warp,
// one a query tile, 1.46 ms, as the tiles then run in step and neither covers
// the other's softmax.
#include <cuda_bf16.h>

#include <cmath>

#include "internal.h"
#include "latent.h"
#include "latent_map.h"
#include "latent_mma.cuh"

namespace dsaidx {

namespace {

constexpr int kNope = IDX_EXPANDED_NOPE_DIM, kPe = IDX_LATENT_PE_DIM, kVal = IDX_EXPANDED_V_DIM;
constexpr int kTile = 128;                  // queries of a tile, keys of a tile
constexpr int kUnit = 16384;                // bytes of a ring unit
constexpr int kUnits = 8;
constexpr int kExpThreads = 384;
constexpr int kSoftThreads = 128;           // of one query tile
constexpr float kNone = -3.0e38f;           // maximum of a row without a key so far
constexpr float kGrow = 8.0f;               // log2 by which a score may pass the maximum

constexpr int kQOff = 0;                                 // two tiles of three chunks
constexpr int kRingOff = 2 * 3 * kUnit;
constexpr int kBarOff = kRingOff + kUnits * kUnit;
constexpr int kSmem = kBarOff + 256 + 1024;
static_assert(kSmem <= 232448, "fits one SM's shared memory");

struct Params {
    const int32_t* cu_q;
    const int32_t* cu_k;
    int batch, heads;
    int64_t total_q, total_k;
    int q_swap, kn_swap, kp_swap, v_swap;
    int kn_one, v_one;           // keys / values shared by the heads: head coordinate 0
    int fold;                    // a CTA takes the j-th query tile from either end of its sequence
    float scale_log2;
    __nv_bfloat16* out;
    float* lse;
    int32_t* status;
};

// The queries of a CTA: two tiles of a sequence whose queries are rows
// q0 .. q0 + nq and whose keys are rows k0 .. k0 + nk.  Tile t begins at its
// query off[t] (off1 < 0: one tile); query r sees keys 0 .. nk - nq + r.
struct Item {
    int q0, nq, k0, nk, off0, off1;
};

// Block `block` counted from the last sequence's last block down (later blocks
// of a sequence see more keys and start first).  False: there are fewer.
// Executed by a whole warp.
__device__ bool find_item(const Params& p, int block, Item& it) {
    const int lane = lane_id();
    int left = block;
    for (int b1 = p.batch; b1 > 0; b1 -= 32) {
        const int b = b1 - 1 - lane;
        int n = 0, q0 = 0, q1 = 0, k0 = 0, k1 = 0;
        if (b >= 0) {
            q0 = __ldg(p.cu_q + b), q1 = __ldg(p.cu_q + b + 1), k0 = __ldg(p.cu_k + b), k1 = __ldg(p.cu_k + b + 1);
            if (q0 < 0 || q1 < q0 || q1 > p.total_q || k0 < 0 || k1 < k0 || k1 > p.total_k)
                set_status(p.status, IDX_ERR_DEVICE_CHECK);
            else
                n = (q1 - q0 + 2 * kTile - 1) / (2 * kTile);
        }
        int v = n;
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(~0u, v, d);
            if (lane >= d) v += u;
        }
        const unsigned in = __ballot_sync(~0u, left < v);
        if (in) {
            const int src = __ffs(in) - 1;
            q0 = __shfl_sync(~0u, q0, src), q1 = __shfl_sync(~0u, q1, src);
            k0 = __shfl_sync(~0u, k0, src), k1 = __shfl_sync(~0u, k1, src);
            const int before = __shfl_sync(~0u, v - n, src);
            n = __shfl_sync(~0u, n, src);
            const int qb = n - 1 - (left - before);
            it.q0 = q0;
            it.nq = q1 - q0;
            it.k0 = k0;
            it.nk = k1 - k0;
            const int tiles = (it.nq + kTile - 1) / kTile;
            const int t0 = p.fold ? qb : 2 * qb, t1 = p.fold ? tiles - 1 - qb : 2 * qb + 1;
            it.off0 = t0 * kTile;
            it.off1 = t1 > t0 && t1 < tiles ? t1 * kTile : -1;
            return true;
        }
        left -= __shfl_sync(~0u, v, 31);
    }
    return false;
}

__device__ __forceinline__ void tmem_ld32_nowait(uint32_t taddr, uint32_t (&a)[16], uint32_t (&b)[16]) {
    tmem_ld16_nowait(taddr, a);
    tmem_ld16_nowait(taddr + 16, b);
}

__global__ void __launch_bounds__(kExpThreads, 1)
    expanded_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap kn_map,
                    const __grid_constant__ CUtensorMap kp_map, const __grid_constant__ CUtensorMap v_map,
                    const Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + kBarOff);   // [2], by tile parity
    uint64_t* v_full = k_full + 2;     // [2]
    uint64_t* k_done = k_full + 4;     // [2] both score products of a tile have read its keys
    uint64_t* v_done = k_full + 6;     // [2]
    uint64_t* s_full = k_full + 8;     // [2], by query tile
    uint64_t* pv_done = k_full + 10;   // [2]
    uint64_t* q_full = k_full + 12;
    uint64_t* v_clean = k_full + 13;
    uint64_t* v_tail = k_full + 14;    // the last tile's values are on their way
    uint64_t* drain = k_full + 15;
    uint64_t* p_full = k_full + 16;    // [2]
    uint32_t* sh_tmem = reinterpret_cast<uint32_t*>(k_full + 18);
    int* sh_abort = reinterpret_cast<int*>(k_full + 19);
    int* sh_item = reinterpret_cast<int*>(k_full + 20);   // found, then the item (6 values)
    const int warp = warp_id(), lane = lane_id();
    const int h = blockIdx.x % p.heads, block = blockIdx.x / p.heads;

    if (warp == 0 && elect_one()) {
        for (int i = 0; i < 16; ++i) mbar_init(k_full + i, 1);
        mbar_init(p_full, kSoftThreads);
        mbar_init(p_full + 1, kSoftThreads);
        *sh_abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(sh_tmem, 512);
        tmem_relinquish();
        if (elect_one()) {
            tma_prefetch_desc(&q_map);
            tma_prefetch_desc(&kn_map);
            tma_prefetch_desc(&kp_map);
            tma_prefetch_desc(&v_map);
        }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (warp == 2) {
        Item it{};
        const bool found = find_item(p, block, it);
        if (lane == 0) {
            sh_item[0] = found;
            sh_item[1] = it.q0;
            sh_item[2] = it.nq;
            sh_item[3] = it.k0;
            sh_item[4] = it.nk;
            sh_item[5] = it.off0;
            sh_item[6] = it.off1;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *sh_tmem;
    volatile int* abort_flag = sh_abort;
    const bool found = sh_item[0] != 0;
    const Item w{sh_item[1], sh_item[2], sh_item[3], sh_item[4], sh_item[5], sh_item[6]};
    // key tiles of the two query tiles: up to the last query's horizon
    const bool two = w.off1 >= 0;
    auto horizon = [&](int off) { return max(0, min(w.nk, w.nk - w.nq + min(w.nq, off + kTile))); };
    const int vis0 = horizon(w.off0), vis1 = two ? horizon(w.off1) : 0;
    const int n0 = found ? (vis0 + kTile - 1) / kTile : 0, n1 = found ? (vis1 + kTile - 1) / kTile : 0;
    const int n = max(n0, n1);
    // the last tile reaches behind the sequence's keys
    const bool tail = n * kTile > w.nk;

    if (warp == 1) {
        // ---- loads ----
        if (n > 0 && elect_one()) {
            mbar_arrive_expect_tx(q_full, (two ? 6 : 3) * kUnit);
            for (int t = 0; t < (two ? 2 : 1); ++t)
                for (int c = 0; c < 3; ++c) {
                    const int row = w.q0 + (t ? w.off1 : w.off0);
                    tma_tile_3d(smem_u32(smem + kQOff) + (3 * t + c) * kUnit, &q_map, q_full, 64 * c, p.q_swap ? row : h,
                                p.q_swap ? h : row);
                }
            const int hk = p.kn_one ? 0 : h, hv = p.v_one ? 0 : h;
            const uint32_t ring = smem_u32(smem + kRingOff);
            bool ok = true;
            int i = 0;
            for (; i < n; ++i) {
                const int row = w.k0 + i * kTile, u = 5 * i;
                auto unit = [&](int c) { return ring + ((u + c) % kUnits) * kUnit; };
                // (of tile i - 2)
                if (i >= 2 && !(ok = mbar_wait(v_done + (i & 1), ((i >> 1) & 1) ^ 1, p.status, abort_flag))) break;
                uint64_t* full = k_full + (i & 1);
                mbar_arrive_expect_tx(full, 3 * kUnit);
                for (int c = 0; c < 2; ++c)
                    tma_tile_3d(unit(c), &kn_map, full, 64 * c, p.kn_swap ? row : hk, p.kn_swap ? hk : row);
                tma_tile_3d(unit(2), &kp_map, full, 0, p.kp_swap ? row : 0, p.kp_swap ? 0 : row);
                // (of tile i - 1)
                if (i >= 1 && !(ok = mbar_wait(k_done + ((i - 1) & 1), ((i - 1) >> 1) & 1, p.status, abort_flag))) break;
                full = v_full + (i & 1);
                mbar_arrive_expect_tx(full, 2 * kUnit);
                for (int c = 0; c < 2; ++c) {
                    const int r = row + 64 * c;
                    tma_tile_3d(unit(3 + c), &v_map, full, 0, p.v_swap ? r : hv, p.v_swap ? hv : r);
                    tma_tile_3d(unit(3 + c) + kUnit / 2, &v_map, full, 64, p.v_swap ? r : hv, p.v_swap ? hv : r);
                }
            }
            if (ok) mbar_arrive(v_tail);
            // copies in flight land before the CTA leaves
            mbar_wait(q_full, 0, p.status, nullptr);
            for (int j = i > 1 ? i - 2 : 0; j <= i; ++j) {
                if (j < n && (j < i || !ok)) mbar_wait(k_full + (j & 1), (j >> 1) & 1, p.status, nullptr);
                if (j < i) mbar_wait(v_full + (j & 1), (j >> 1) & 1, p.status, nullptr);
            }
        }
    } else if (warp == 0) {
        // ---- every MMA ----
        if (n > 0 && elect_one()) {
            constexpr uint32_t kIdS = idesc_bf16(kTile, kTile, false, false);
            constexpr uint32_t kIdO = idesc_bf16(kTile, kVal, false, true);
            const uint32_t ring = smem_u32(smem + kRingOff), q_addr = smem_u32(smem + kQOff);
            const int last = two ? 1 : 0;      // the tile that reads a unit last
            auto scores = [&](int t, int i) {
#pragma unroll 1
                for (int c = 0; c < 3; ++c) {
                    const uint32_t unit = ring + ((5 * i + c) % kUnits) * kUnit;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_bf16(tmem + t * kTile, sdesc_sw128(q_addr + (3 * t + c) * kUnit + 32 * k),
                                 sdesc_sw128(unit + 32 * k), kIdS, (c | k) != 0 ? 1u : 0u);
                }
                if (t == last) mma_commit(k_done + (i & 1));
                mma_commit(s_full + t);
            };
            auto values = [&](int t, int i) -> bool {
                if (!mbar_wait(p_full + t, i & 1, p.status, abort_flag)) return false;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const uint32_t unit = ring + ((5 * i + 3 + c) % kUnits) * kUnit;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_bf16_ts(tmem + (2 + t) * kTile, tmem + t * kTile + 32 * c + 8 * k,
                                    sdesc_mn_sw128(unit + 2048 * k, kUnit / 2), kIdO, (i | c | k) != 0 ? 1u : 0u);
                }
                if (t == last) mma_commit(v_done + (i & 1));
                mma_commit(pv_done + t);
                return true;
            };
            // a key tile's copies are waited for once, by the query tile that
            // comes first
            auto keys_in = [&](int i) -> bool {
                if (!mbar_wait(k_full + (i & 1), (i >> 1) & 1, p.status, abort_flag)) return false;
                tc_fence_after();
                return true;
            };
            bool ok = mbar_wait(q_full, 0, p.status, abort_flag) && keys_in(0);
            if (ok) {
                if (n0 > 0) scores(0, 0);
                if (n1 > 0) scores(1, 0);
            }
            for (int i = 0; i < n && ok; ++i) {
                ok = mbar_wait(v_full + (i & 1), (i >> 1) & 1, p.status, abort_flag);
                if (ok && tail && i == n - 1) ok = mbar_wait(v_clean, 0, p.status, abort_flag);
                if (ok && i < n0) ok = values(0, i);
                if (ok && i + 1 < n0) {
                    ok = keys_in(i + 1);
                    if (ok) scores(0, i + 1);
                }
                if (ok && i < n1) ok = values(1, i);
                if (ok && i + 1 < n1) {
                    if (i + 1 >= n0) ok = keys_in(i + 1);
                    if (ok) scores(1, i + 1);
                }
            }
            mma_commit(drain);
            mbar_wait(drain, 0, p.status, nullptr);
        }
    } else if (warp == 2) {
        // ---- zeroes behind the last key ----
        if (tail && n > 0) {
            const int keep = w.nk - (n - 1) * kTile;      // rows of the last tile that hold keys
            // only then are the units' earlier uses over and their parity tells
            bool ok = mbar_wait(v_tail, 0, p.status, abort_flag);
            ok = ok && mbar_wait(v_full + ((n - 1) & 1), ((n - 1) >> 1) & 1, p.status, abort_flag);
            for (int c = 0; c < 2 && ok; ++c) {
                uint4* unit = reinterpret_cast<uint4*>(smem + kRingOff + (5 * (n - 1) + 3 + c) % kUnits * kUnit);
                for (int r = max(0, keep - 64 * c); r < 64; ++r)
                    if (lane < 16) unit[(lane >> 3) * 512 + r * 8 + (lane & 7)] = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(v_clean);
        }
    } else if (warp >= 4 && found && (warp < 8 || two)) {
        // ---- softmax of tile t, one query a thread ----
        const int t = (warp - 4) >> 2, sw = warp & 3;
        const int nt = t ? n1 : n0, off = (t ? w.off1 : w.off0) + 32 * sw, row = off + lane;   // query of the sequence
        const uint32_t lanes = static_cast<uint32_t>(32 * sw) << 16;
        const uint32_t s_col = tmem + lanes + t * kTile, o_col = tmem + lanes + (2 + t) * kTile;
        const int see = min(w.nk, w.nk - w.nq + row + 1);      // keys this query sees (may be <= 0)
        // all 32 queries of the warp see this many
        const int see_all = min(w.nk, w.nk - w.nq + off + 1);
        float m = kNone, l = 0.0f;
        bool ok = true;
        const unsigned long long sc2 = f2_pack(p.scale_log2, p.scale_log2), one2 = f2_pack(1.0f, 1.0f);
        for (int i = 0; i < nt; ++i) {
            ok = mbar_wait(s_full + t, i & 1, p.status, abort_flag);
            if (!__all_sync(~0u, ok)) { ok = false; break; }
            tc_fence_after();
            const bool cut = see_all < (i + 1) * kTile;     // (uniform) some key of the tile is masked
            const int lim = see - i * kTile;
            uint32_t pk[64];
            float ls = 0.0f;
            // weights and their sum under maximum m; the largest exponent
            auto weights = [&]() -> float {
                const unsigned long long nm2 = f2_pack(-m, -m);
                unsigned long long sum2 = f2_pack(0.0f, 0.0f);
                float top = kNone;
                uint32_t a[2][16], b[2][16];
                tmem_ld32_nowait(s_col, a[0], b[0]);
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    tmem_wait_ld16(a[g & 1]);
                    tmem_wait_ld16(b[g & 1]);
                    if (g < 3) tmem_ld32_nowait(s_col + 32 * (g + 1), a[(g + 1) & 1], b[(g + 1) & 1]);
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const uint32_t s0 = j < 16 ? a[g & 1][j] : b[g & 1][j - 16];
                        const uint32_t s1 = j < 16 ? a[g & 1][j + 1] : b[g & 1][j - 15];
                        float2 y = f2_unpack(f2_fma(f2_pack(__uint_as_float(s0), __uint_as_float(s1)), sc2, nm2));
                        if (cut) {
                            if (32 * g + j >= lim) y.x = -INFINITY;
                            if (32 * g + j + 1 >= lim) y.y = -INFINITY;
                        }
                        top = max3(top, y.x, y.y);
                        y.x = exp2_fast(y.x);
                        y.y = exp2_fast(y.y);
                        sum2 = f2_fma(f2_pack(y.x, y.y), one2, sum2);
                        pk[16 * g + j / 2] = bf16x2(y.x, y.y);
                    }
                }
                const float2 s = f2_unpack(sum2);
                ls = s.x + s.y;
                return top;
            };
            bool grow = true;
            if (i > 0) {
                if (!__all_sync(~0u, mbar_wait(pv_done + t, (i - 1) & 1, p.status, abort_flag))) { ok = false; break; }
                grow = weights() > kGrow;
            }
            if (__any_sync(~0u, grow)) {
                // move the maximum: over the tile's visible scores
                float v = kNone;
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                    uint32_t a[16];
                    tmem_ld16_nowait(s_col + 16 * g, a);
                    tmem_wait_ld16(a);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (!cut || 16 * g + j < lim) v = fmaxf(v, __uint_as_float(a[j]) * p.scale_log2);
                }
                v = fmaxf(v, m);
                const float f = exp2_fast(m - v);
                m = v;
                l *= f;
                if (i > 0) {
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < kVal; c += 16) {
                        uint32_t a[16];
                        tmem_ld16_nowait(o_col + c, a);
                        tmem_wait_ld16(a);
#pragma unroll
                        for (int j = 0; j < 16; ++j) a[j] = __float_as_uint(__uint_as_float(a[j]) * f);
                        tmem_st16(o_col + c, a);
                    }
                }
                weights();
            }
            l += ls;
#pragma unroll
            for (int g = 0; g < 4; ++g) tmem_st16(s_col + 16 * g, *reinterpret_cast<const uint32_t(*)[16]>(pk + 16 * g));
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(p_full + t);
        }
        if (nt > 0 && ok) ok = __all_sync(~0u, mbar_wait(pv_done + t, (nt - 1) & 1, p.status, abort_flag));
        if (ok && row < w.nq) {
            const int64_t at = static_cast<int64_t>(w.q0 + row) * p.heads + h;
            if (p.lse != nullptr) p.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
        }
        if (ok) {
            tc_fence_after();
            const float f = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
            uint4* dst = reinterpret_cast<uint4*>(p.out + (static_cast<int64_t>(w.q0 + row) * p.heads + h) * kVal);
#pragma unroll
            for (int c = 0; c < kVal; c += 16) {
                uint32_t a[16];
                if (nt > 0) {
                    tmem_ld16_nowait(o_col + c, a);
                    tmem_wait_ld16(a);
                }
                uint32_t o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    o[j] = nt > 0 ? bf16x2(__uint_as_float(a[2 * j]) * f, __uint_as_float(a[2 * j + 1]) * f) : 0u;
                if (row < w.nq) {
                    dst[c / 8] = make_uint4(o[0], o[1], o[2], o[3]);
                    dst[c / 8 + 1] = make_uint4(o[4], o[5], o[6], o[7]);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

}  // namespace

cudaError_t launch_expanded(const ExpandedArgs& a, int sms, cudaStream_t st) {
    EncodeTiledFn enc = encode_tiled_fn();
    if (!enc) return cudaErrorNotSupported;
    Params p{};
    p.cu_q = a.cu_q; p.cu_k = a.cu_k; p.batch = a.batch; p.heads = a.heads;
    p.total_q = a.total_q; p.total_k = a.total_k;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.out = static_cast<__nv_bfloat16*>(a.out); p.lse = a.lse; p.status = a.status;
    p.kn_one = a.kn_head == 0; p.v_one = a.v_head == 0;
    CUtensorMap q, kn, kp, v;
    // without keys nothing is loaded; the maps then only have to be valid
    const int64_t rows = a.total_k > 0 ? a.total_k : 1;
    const void* kn_p = a.total_k > 0 ? a.kn : a.q;
    const void* kp_p = a.total_k > 0 ? a.kp : a.q;
    const void* v_p = a.total_k > 0 ? a.v : a.q;
    const int kn_heads = p.kn_one ? 1 : a.heads, v_heads = p.v_one ? 1 : a.heads;
    if (!head_map(&q, enc, a.q, kNope + kPe, a.q_row, a.q_head, a.total_q, a.heads, 1, kTile, &p.q_swap) ||
        !head_map(&kn, enc, kn_p, kNope, a.kn_row, a.kn_head, rows, kn_heads, 1, kTile, &p.kn_swap) ||
        !head_map(&kp, enc, kp_p, kPe, a.kp_row, kPe, rows, 1, 1, kTile, &p.kp_swap) ||
        !head_map(&v, enc, v_p, kVal, a.v_row, a.v_head, rows, v_heads, 1, kTile / 2, &p.v_swap))
        return cudaErrorInvalidValue;
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = set_smem_once(expanded_kernel, kSmem, done);
    if (e != cudaSuccess) return e;
    // Where no CTA would wait for an SM, the longest one decides: a sequence's
    // first and last tile together, second and last but one, and so on.
    p.fold = a.total_q * a.heads <= static_cast<int64_t>(2 * kTile) * sms;
    // at most one partly filled block of queries a sequence
    const int64_t blocks = (a.total_q + 2 * kTile - 1) / (2 * kTile) + a.batch - 1;
    if (blocks * a.heads >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks * a.heads), 1, 1);
    cfg.blockDim = dim3(kExpThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    kt_mark(st);
    e = cudaLaunchKernelEx(&cfg, expanded_kernel, q, kn, kp, v, p);
    kt_mark(st);
    return e;
}

}  // namespace dsaidx
