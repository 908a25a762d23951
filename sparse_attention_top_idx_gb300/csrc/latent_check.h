// latent_check.h -- argument checks shared by the C entries of the latent
// attention over either kind of record (host only).
#pragma once

#include <cmath>

#include "internal.h"
#include "latent.h"

namespace dsaidx {

inline bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline bool mult8(int64_t s) { return s % 8 == 0; }

constexpr int64_t kInt31 = int64_t(1) << 31;

// Number of SMs of the current device, asked for once a device.
inline bool sm_count(int* sms) {
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const bool kept = dev >= 0 && dev < 64;
    if (kept && (*sms = known[dev].load(std::memory_order_relaxed)) > 0) return true;
    if (cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return false;
    if (kept) known[dev].store(*sms, std::memory_order_relaxed);
    return true;
}

inline bool pool_ok(const idx_latent_pool* p) {
    if (!p || !p->data_dev || !aligned(p->data_dev, 128)) return false;
    if (p->block_size < 1 || p->block_size > 65536 || p->num_blocks < 1 || p->num_blocks >= kInt31) return false;
    return p->num_blocks * p->block_size < kInt31;
}

inline idx_status status_of(cudaError_t e) { return e == cudaSuccess ? IDX_OK : IDX_ERR_CUDA; }

// What the absorbed calls check alike; ws_need: bytes the call itself uses.
inline idx_status attend_check(const idx_latent_pool* pool, const void* ql, int64_t ql_row, int64_t ql_head,
                               const void* qp, int64_t qp_row, int64_t qp_head, int64_t rows, int heads,
                               int64_t max_keys, int64_t keys_cap, float scale, const void* out, const void* ws,
                               size_t ws_bytes, bool paged, size_t (*ws_need)(int64_t, int, int64_t, bool)) {
    if (!pool_ok(pool) || rows < 0 || heads < 1 || heads > IDX_LATENT_MAX_HEADS || max_keys < 0 || max_keys > keys_cap)
        return IDX_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return IDX_ERR_INVALID_ARG;
    if (rows >= kInt31 || rows * ((heads + 63) / 64) >= kInt31) return IDX_ERR_INVALID_ARG;
    if (rows == 0) return IDX_OK;
    if (!ql || !qp || !out || !ws) return IDX_ERR_INVALID_ARG;
    if (!aligned(ql, 16) || !aligned(qp, 16) || !aligned(out, 16) || !aligned(ws, 256)) return IDX_ERR_INVALID_ARG;
    if (!mult8(ql_row) || !mult8(ql_head) || !mult8(qp_row) || !mult8(qp_head)) return IDX_ERR_INVALID_ARG;
    // strides that are stepped over: positive and within a tensor map's range
    const int64_t cap = int64_t(1) << 38;
    if (rows > 1 && (ql_row < 1 || ql_row > cap || qp_row < 1 || qp_row > cap)) return IDX_ERR_INVALID_ARG;
    if (heads > 1 && (ql_head < 1 || ql_head > cap || qp_head < 1 || qp_head > cap)) return IDX_ERR_INVALID_ARG;
    if (ws_bytes < ws_need(rows, heads, max_keys, paged)) return IDX_ERR_WORKSPACE_TOO_SMALL;
    return IDX_OK;
}

}  // namespace dsaidx
