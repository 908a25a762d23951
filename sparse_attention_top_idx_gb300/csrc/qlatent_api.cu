// qlatent_api.cu -- the C ABI of the 8-bit latent cache (declared in
// include/dsaidx_qlatent.h): argument checks and dispatch.  No device memory is
// allocated and no stream synchronised.
#include "latent_check.h"
#include "qlatent.h"

using namespace dsaidx;

namespace {

// Records begin at multiples of 128 bytes, which the kernels count in 32 bits.
bool qpool_ok(const idx_latent_pool* p) {
    return pool_ok(p) && p->num_blocks <= IDX_QLATENT_MAX_POOL_BYTES / qlatent_block_bytes(p->block_size);
}

}  // namespace

extern "C" {

size_t idx_qlatent_block_bytes(int block_size) {
    if (block_size < 1 || block_size > 65536) return 0;
    return static_cast<size_t>(qlatent_block_bytes(block_size));
}

idx_status idx_qlatent_append(const idx_latent_pool* pool, const void* latent_dev, int64_t latent_stride,
                              const void* pe_dev, int64_t pe_stride, const int64_t* positions_dev,
                              const int64_t* slot_mapping_dev, int64_t n, const uint64_t* steps_dev, float amplitude,
                              unsigned flags, int32_t* status_dev, void* stream) {
    if (!qpool_ok(pool) || n < 0 || (flags & ~IDX_ROPE_HALF) != 0u) return IDX_ERR_INVALID_ARG;
    if (n == 0) return IDX_OK;
    if (!latent_dev || !pe_dev || !slot_mapping_dev || (steps_dev && !positions_dev)) return IDX_ERR_INVALID_ARG;
    if (!aligned(latent_dev, 16) || !aligned(pe_dev, 16) || !mult8(latent_stride) || !mult8(pe_stride) ||
        !aligned(slot_mapping_dev, 8) || !aligned(positions_dev, 8) || !aligned(steps_dev, 8) || !aligned(status_dev, 4))
        return IDX_ERR_INVALID_ARG;
    if ((n + 3) / 4 >= kInt31) return IDX_ERR_INVALID_ARG;
    QAppendArgs a{{latent_dev, pe_dev, pool->data_dev, positions_dev, slot_mapping_dev, steps_dev, latent_stride,
                   pe_stride, n, pool->num_blocks * pool->block_size, amplitude, flags, status_dev},
                  pool->block_size, qlatent_block_bytes(pool->block_size)};
    return status_of(launch_qappend(a, static_cast<cudaStream_t>(stream)));
}

idx_status idx_qlatent_read(const idx_latent_pool* pool, const int64_t* slots_dev, int64_t n, void* out_dev,
                            int64_t out_stride, int32_t* status_dev, void* stream) {
    if (!qpool_ok(pool) || n < 0 || (n + 3) / 4 >= kInt31 || out_stride < IDX_LATENT_RECORD || !mult8(out_stride))
        return IDX_ERR_INVALID_ARG;
    if (n == 0) return IDX_OK;
    if (!slots_dev || !out_dev || !aligned(slots_dev, 8) || !aligned(out_dev, 16) || !aligned(status_dev, 4))
        return IDX_ERR_INVALID_ARG;
    QReadArgs a{pool->data_dev, slots_dev, out_dev, n, out_stride, pool->num_blocks * pool->block_size,
                qlatent_block_bytes(pool->block_size), pool->block_size, status_dev};
    return status_of(launch_qread(a, static_cast<cudaStream_t>(stream)));
}

idx_status idx_qlatent_attend_slots(const idx_latent_pool* pool, const void* ql_dev, int64_t ql_row_stride,
                                    int64_t ql_head_stride, const void* qp_dev, int64_t qp_row_stride,
                                    int64_t qp_head_stride, const int64_t* slots_dev, int64_t slots_stride,
                                    int64_t rows, int heads, int topk, float scale, void* out_dev, float* lse_dev,
                                    void* workspace_dev, size_t ws_bytes, void* stream) {
    if (!qpool_ok(pool)) return IDX_ERR_INVALID_ARG;
    const idx_status c = attend_check(pool, ql_dev, ql_row_stride, ql_head_stride, qp_dev, qp_row_stride,
                                      qp_head_stride, rows, heads, topk, int64_t(1) << 24, scale, out_dev,
                                      workspace_dev, ws_bytes, false, qattend_ws_need);
    if (c != IDX_OK || rows == 0) return c;
    if ((!slots_dev && topk > 0) || !aligned(slots_dev, 8) || !aligned(lse_dev, 4)) return IDX_ERR_INVALID_ARG;
    AttendArgs a{};
    a.ql = ql_dev; a.qp = qp_dev;
    a.ql_row = ql_row_stride; a.ql_head = ql_head_stride; a.qp_row = qp_row_stride; a.qp_head = qp_head_stride;
    a.pool = pool->data_dev; a.num_slots = pool->num_blocks * pool->block_size; a.block_size = pool->block_size;
    a.slots = slots_dev; a.slots_stride = slots_stride;
    a.rows = rows; a.heads = heads; a.max_keys = topk; a.scale = scale;
    a.out = out_dev; a.lse = lse_dev;
    a.status = static_cast<int32_t*>(workspace_dev);
    a.ws = static_cast<uint8_t*>(workspace_dev) + 256;
    return status_of(launch_qattend(a, qlatent_block_bytes(pool->block_size), static_cast<cudaStream_t>(stream)));
}

idx_status idx_qlatent_attend_paged(const idx_latent_pool* pool, const void* ql_dev, int64_t ql_row_stride,
                                    int64_t ql_head_stride, const void* qp_dev, int64_t qp_row_stride,
                                    int64_t qp_head_stride, const int32_t* block_table_dev, int max_blocks_per_seq,
                                    const int32_t* seq_lens_dev, int batch, int max_seq_len, int heads, float scale,
                                    void* out_dev, float* lse_dev, void* workspace_dev, size_t ws_bytes,
                                    void* stream) {
    if (max_blocks_per_seq < 1) return IDX_ERR_INVALID_ARG;
    if (!qpool_ok(pool)) return IDX_ERR_INVALID_ARG;
    const idx_status c = attend_check(pool, ql_dev, ql_row_stride, ql_head_stride, qp_dev, qp_row_stride,
                                      qp_head_stride, batch, heads, max_seq_len, kInt31 - 256, scale, out_dev,
                                      workspace_dev, ws_bytes, true, qattend_ws_need);
    if (c != IDX_OK || batch == 0) return c;
    if (!block_table_dev || !seq_lens_dev || !aligned(block_table_dev, 4) || !aligned(seq_lens_dev, 4) ||
        !aligned(lse_dev, 4))
        return IDX_ERR_INVALID_ARG;
    AttendArgs a{};
    a.ql = ql_dev; a.qp = qp_dev;
    a.ql_row = ql_row_stride; a.ql_head = ql_head_stride; a.qp_row = qp_row_stride; a.qp_head = qp_head_stride;
    a.pool = pool->data_dev; a.num_slots = pool->num_blocks * pool->block_size; a.block_size = pool->block_size;
    a.block_table = block_table_dev; a.seq_lens = seq_lens_dev; a.mbps = max_blocks_per_seq;
    a.rows = batch; a.heads = heads; a.max_keys = max_seq_len; a.scale = scale;
    a.out = out_dev; a.lse = lse_dev;
    a.status = static_cast<int32_t*>(workspace_dev);
    a.ws = static_cast<uint8_t*>(workspace_dev) + 256;
    return status_of(launch_qattend(a, qlatent_block_bytes(pool->block_size), static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
