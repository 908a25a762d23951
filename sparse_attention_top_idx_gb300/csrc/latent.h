// latent.h -- host structures shared by the latent-attention C ABI layer
// (latent_api.cu) and its kernels.  Not part of the public interface.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "dsaidx_latent.h"

namespace dsaidx {

struct RopeArgs {
    const void* x;
    void* y;
    const int64_t* positions;
    const uint64_t* steps;
    int64_t xt, xh, yt, yh, tokens;
    int dtype, heads, head_dim, rot, offset;
    float amplitude;
    unsigned flags;
};
cudaError_t launch_rope(const RopeArgs& a, int sms, cudaStream_t st);

struct AppendArgs {
    const void* latent;
    const void* pe;
    void* pool;
    const int64_t* positions;
    const int64_t* slots;
    const uint64_t* steps;     // null: no rotation
    int64_t latent_stride, pe_stride, n, num_slots;
    float amplitude;
    unsigned flags;
    int32_t* status;
};
cudaError_t launch_append(const AppendArgs& a, cudaStream_t st);

// Absorbed attention: one row = one query of every head.  Keys come from a
// slot list (block_table null) or from a paged context.
struct AttendArgs {
    const void* ql;
    const void* qp;
    int64_t ql_row, ql_head, qp_row, qp_head;
    const void* pool;
    int64_t num_slots;
    int block_size;
    const int64_t* slots;
    int64_t slots_stride;
    const int32_t* block_table;
    const int32_t* seq_lens;
    int64_t rows;
    int mbps, heads, max_keys;   // topk or max_seq_len
    float scale;
    void* out;
    float* lse;
    int32_t* status;
    void* ws;                    // behind the header
};
cudaError_t launch_attend(const AttendArgs& a, cudaStream_t st);
size_t attend_ws_bytes(int64_t rows, int heads, int64_t max_keys);              // of this call and every smaller one
size_t attend_ws_need(int64_t rows, int heads, int64_t max_keys, bool paged);   // of this call

struct ExpandedArgs {
    const void* q;
    const void* kn;
    const void* kp;
    const void* v;
    int64_t q_row, q_head, kn_row, kn_head, kp_row, v_row, v_head, total_q, total_k;
    const int32_t* cu_q;
    const int32_t* cu_k;
    int batch, heads;
    float scale;
    void* out;
    float* lse;
    int32_t* status;
};
cudaError_t launch_expanded(const ExpandedArgs& a, int sms, cudaStream_t st);

}  // namespace dsaidx
