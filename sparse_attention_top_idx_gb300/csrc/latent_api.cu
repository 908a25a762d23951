// latent_api.cu -- the C ABI of the latent attention (declared in
// include/dsaidx_latent.h): argument checks and dispatch.  No device memory
// is allocated and no stream synchronised.
#include <cmath>

#include "latent.h"
#include "latent_check.h"
#include "strides.h"

using namespace dsaidx;

extern "C" {

idx_status idx_rope_steps(int rot_dim, double base, int scaling, double factor, double original_max_pos,
                          double beta_fast, double beta_slow, uint64_t* steps_host, float* amplitude_out) {
    if (!steps_host || !amplitude_out || rot_dim < 2 || rot_dim > IDX_ROPE_MAX_DIM || rot_dim % 2)
        return IDX_ERR_INVALID_ARG;
    if (!(base > 1.0) || !std::isfinite(base) || scaling < IDX_ROPE_NONE || scaling > IDX_ROPE_YARN)
        return IDX_ERR_INVALID_ARG;
    if (scaling != IDX_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return IDX_ERR_INVALID_ARG;
    if (scaling == IDX_ROPE_YARN && (!(original_max_pos >= 1.0) || !std::isfinite(original_max_pos) ||
                                     !(beta_slow > 0.0) || !(beta_fast >= beta_slow) || !std::isfinite(beta_fast)))
        return IDX_ERR_INVALID_ARG;
    const double kPi = 3.14159265358979323846;
    double low = 0.0, high = 0.0;
    if (scaling == IDX_ROPE_YARN) {
        const double per = rot_dim / (2.0 * std::log(base));
        low = std::fmax(std::floor(per * std::log(original_max_pos / (beta_fast * 2.0 * kPi))), 0.0);
        high = std::fmin(std::ceil(per * std::log(original_max_pos / (beta_slow * 2.0 * kPi))), rot_dim - 1.0);
    }
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot_dim);
        if (scaling == IDX_ROPE_LINEAR) f /= factor;
        if (scaling == IDX_ROPE_YARN) {
            const double r = std::fmin(std::fmax((i - low) / std::fmax(high - low, 0.001), 0.0), 1.0);
            f = f * (1.0 - r) + f / factor * r;
        }
        // f <= 1 radian, so the product stays below 2^64
        steps_host[i] = static_cast<uint64_t>(f / (2.0 * kPi) * 0x1p64);
    }
    *amplitude_out = scaling == IDX_ROPE_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
    return IDX_OK;
}

idx_status idx_rope(const void* x_dev, int64_t x_token_stride, int64_t x_head_stride, void* y_dev,
                    int64_t y_token_stride, int64_t y_head_stride, int dtype, int64_t tokens, int heads, int head_dim,
                    const int64_t* positions_dev, const uint64_t* steps_dev, int rot_dim, int offset, float amplitude,
                    unsigned flags, void* stream) {
    if (dtype < IDX_DT_BF16 || dtype > IDX_DT_FP32 || (flags & ~(IDX_ROPE_HALF | IDX_ROPE_TRANSPOSE)) != 0u)
        return IDX_ERR_INVALID_ARG;
    if (tokens < 0 || heads < 1 || heads > IDX_ROPE_MAX_HEADS || head_dim < 1 || head_dim > IDX_ROPE_MAX_DIM)
        return IDX_ERR_INVALID_ARG;
    if (rot_dim < 2 || rot_dim % 2 || offset < 0 || rot_dim > head_dim || offset > head_dim - rot_dim)
        return IDX_ERR_INVALID_ARG;
    if (tokens >= 4 * kInt31 / heads) return IDX_ERR_INVALID_ARG;
    if (tokens == 0) return IDX_OK;
    if (!x_dev || !y_dev || !positions_dev || !steps_dev) return IDX_ERR_INVALID_ARG;
    const uintptr_t esize = dtype == IDX_DT_FP32 ? 4 : 2;
    if (!aligned(x_dev, esize) || !aligned(y_dev, esize) || !aligned(positions_dev, 8) || !aligned(steps_dev, 8))
        return IDX_ERR_INVALID_ARG;
    if (x_dev == y_dev && (x_token_stride != y_token_stride || x_head_stride != y_head_stride))
        return IDX_ERR_INVALID_ARG;
    // what is written must be written once: the turned elements in place, else whole heads
    if (!rows_apart(tokens, heads, x_dev == y_dev ? rot_dim : head_dim, y_token_stride, y_head_stride))
        return IDX_ERR_INVALID_ARG;
    int sms = 0;
    if (!sm_count(&sms)) return IDX_ERR_CUDA;
    RopeArgs a{x_dev, y_dev, positions_dev, steps_dev, x_token_stride, x_head_stride, y_token_stride, y_head_stride,
               tokens, dtype, heads, head_dim, rot_dim, offset, amplitude, flags};
    return status_of(launch_rope(a, sms, static_cast<cudaStream_t>(stream)));
}

idx_status idx_latent_append(const idx_latent_pool* pool, const void* latent_dev, int64_t latent_stride,
                             const void* pe_dev, int64_t pe_stride, const int64_t* positions_dev,
                             const int64_t* slot_mapping_dev, int64_t n, const uint64_t* steps_dev, float amplitude,
                             unsigned flags, int32_t* status_dev, void* stream) {
    if (!pool_ok(pool) || n < 0 || (flags & ~IDX_ROPE_HALF) != 0u) return IDX_ERR_INVALID_ARG;
    if (n == 0) return IDX_OK;
    if (!latent_dev || !pe_dev || !slot_mapping_dev || (steps_dev && !positions_dev)) return IDX_ERR_INVALID_ARG;
    if (!aligned(latent_dev, 16) || !aligned(pe_dev, 16) || !mult8(latent_stride) || !mult8(pe_stride) ||
        !aligned(slot_mapping_dev, 8) || !aligned(positions_dev, 8) || !aligned(steps_dev, 8))
        return IDX_ERR_INVALID_ARG;
    if ((n + 3) / 4 >= kInt31) return IDX_ERR_INVALID_ARG;
    AppendArgs a{latent_dev, pe_dev, pool->data_dev, positions_dev, slot_mapping_dev, steps_dev, latent_stride,
                 pe_stride, n, pool->num_blocks * pool->block_size, amplitude, flags, status_dev};
    return status_of(launch_append(a, static_cast<cudaStream_t>(stream)));
}

size_t idx_latent_workspace_bytes(int64_t rows, int heads, int64_t max_keys) {
    if (rows < 0 || heads < 1 || heads > IDX_LATENT_MAX_HEADS || max_keys < 0 || max_keys >= kInt31) return 0;
    if (rows >= kInt31 || rows * ((heads + 63) / 64) >= kInt31) return 0;
    return attend_ws_bytes(rows, heads, max_keys);
}

idx_status idx_latent_attend_slots(const idx_latent_pool* pool, const void* ql_dev, int64_t ql_row_stride,
                                   int64_t ql_head_stride, const void* qp_dev, int64_t qp_row_stride,
                                   int64_t qp_head_stride, const int64_t* slots_dev, int64_t slots_stride,
                                   int64_t rows, int heads, int topk, float scale, void* out_dev, float* lse_dev,
                                   void* workspace_dev, size_t ws_bytes, void* stream) {
    const idx_status c = attend_check(pool, ql_dev, ql_row_stride, ql_head_stride, qp_dev, qp_row_stride,
                                      qp_head_stride, rows, heads, topk, int64_t(1) << 24, scale, out_dev,
                                      workspace_dev, ws_bytes, false, attend_ws_need);
    if (c != IDX_OK || rows == 0) return c;
    if ((!slots_dev && topk > 0) || !aligned(slots_dev, 8)) return IDX_ERR_INVALID_ARG;
    AttendArgs a{};
    a.ql = ql_dev; a.qp = qp_dev;
    a.ql_row = ql_row_stride; a.ql_head = ql_head_stride; a.qp_row = qp_row_stride; a.qp_head = qp_head_stride;
    a.pool = pool->data_dev; a.num_slots = pool->num_blocks * pool->block_size; a.block_size = pool->block_size;
    a.slots = slots_dev; a.slots_stride = slots_stride;
    a.rows = rows; a.heads = heads; a.max_keys = topk; a.scale = scale;
    a.out = out_dev; a.lse = lse_dev;
    a.status = static_cast<int32_t*>(workspace_dev);
    a.ws = static_cast<uint8_t*>(workspace_dev) + 256;
    return status_of(launch_attend(a, static_cast<cudaStream_t>(stream)));
}

idx_status idx_latent_attend_paged(const idx_latent_pool* pool, const void* ql_dev, int64_t ql_row_stride,
                                   int64_t ql_head_stride, const void* qp_dev, int64_t qp_row_stride,
                                   int64_t qp_head_stride, const int32_t* block_table_dev, int max_blocks_per_seq,
                                   const int32_t* seq_lens_dev, int batch, int max_seq_len, int heads, float scale,
                                   void* out_dev, float* lse_dev, void* workspace_dev, size_t ws_bytes, void* stream) {
    if (max_blocks_per_seq < 1) return IDX_ERR_INVALID_ARG;
    const idx_status c = attend_check(pool, ql_dev, ql_row_stride, ql_head_stride, qp_dev, qp_row_stride,
                                      qp_head_stride, batch, heads, max_seq_len, kInt31 - 256, scale, out_dev,
                                      workspace_dev, ws_bytes, true, attend_ws_need);
    if (c != IDX_OK || batch == 0) return c;
    if (!block_table_dev || !seq_lens_dev || !aligned(block_table_dev, 4) || !aligned(seq_lens_dev, 4))
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
    return status_of(launch_attend(a, static_cast<cudaStream_t>(stream)));
}

idx_status idx_latent_attend_expanded(const void* q_dev, int64_t q_row_stride, int64_t q_head_stride,
                                      const void* kn_dev, int64_t kn_row_stride, int64_t kn_head_stride,
                                      const void* kp_dev, int64_t kp_row_stride, const void* v_dev,
                                      int64_t v_row_stride, int64_t v_head_stride, const int32_t* cu_seqlens_q_dev,
                                      const int32_t* cu_seqlens_k_dev, int batch, int64_t total_q, int64_t total_k,
                                      int heads, float scale, void* out_dev, float* lse_dev, int32_t* status_dev,
                                      void* stream) {
    if (batch < 0 || batch > 4096 || total_q < 0 || total_q >= kInt31 - 256 || total_k < 0 || total_k >= kInt31 - 256 ||
        heads < 1 || heads > IDX_LATENT_MAX_HEADS || !std::isfinite(scale))
        return IDX_ERR_INVALID_ARG;
    if (batch == 0 || total_q == 0) return IDX_OK;
    if (!q_dev || !cu_seqlens_q_dev || !cu_seqlens_k_dev || !out_dev) return IDX_ERR_INVALID_ARG;
    if (total_k > 0 && (!kn_dev || !kp_dev || !v_dev)) return IDX_ERR_INVALID_ARG;
    if (!aligned(q_dev, 16) || !aligned(kn_dev, 16) || !aligned(kp_dev, 16) || !aligned(v_dev, 16) ||
        !aligned(out_dev, 16) || !aligned(cu_seqlens_q_dev, 4) || !aligned(cu_seqlens_k_dev, 4))
        return IDX_ERR_INVALID_ARG;
    const int64_t strides[] = {q_row_stride, q_head_stride, kn_row_stride, kn_head_stride, kp_row_stride,
                               v_row_stride, v_head_stride};
    for (int64_t s : strides)
        if (!mult8(s) || s < 0 || s >= kInt31) return IDX_ERR_INVALID_ARG;
    // keys and values may be shared by the heads (head stride 0); other strides
    // that are stepped over are positive
    if (total_q > 1 && q_row_stride < 1) return IDX_ERR_INVALID_ARG;
    if (heads > 1 && q_head_stride < 1) return IDX_ERR_INVALID_ARG;
    if (total_k > 1 && (kn_row_stride < 1 || kp_row_stride < 1 || v_row_stride < 1)) return IDX_ERR_INVALID_ARG;
    if (((total_q + 255) / 256 + batch) * heads >= kInt31) return IDX_ERR_INVALID_ARG;
    int sms = 0;
    if (!sm_count(&sms)) return IDX_ERR_CUDA;
    ExpandedArgs a{q_dev, kn_dev, kp_dev, v_dev, q_row_stride, q_head_stride, kn_row_stride, kn_head_stride,
                   kp_row_stride, v_row_stride, v_head_stride, total_q, total_k, cu_seqlens_q_dev, cu_seqlens_k_dev,
                   batch, heads, scale, out_dev, lse_dev, status_dev};
    return status_of(launch_expanded(a, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
