/*
 * dsaidx_latent.h -- C ABI of libdsaidx's latent attention: what follows the
 * indexer's selection in one sparse-attention layer.
 *
 * The indexer (dsaidx.h) returns the pool slots of the best keys of each
 * query.  The calls here turn queries and keys by their positions, append a
 * token's latent record to a paged cache and attend over the selected records
 * (or over a whole paged context, or over a prompt's expanded keys):
 *
 *   record[slot]  = [ c (512) | p (64) ]                     bf16, 1152 bytes
 *   s[t, h, j]    = scale * (ql[t, h] . c_j + qp[t, h] . p_j)
 *   out[t, h]     = sum_j softmax_j(s) c_j        lse[t, h] = ln sum_j exp s
 *
 * c is the one vector a token's keys and values share (latent attention in
 * its absorbed form: ql is the query already multiplied with the key
 * up-projection, and the caller multiplies out with the value up-projection);
 * p is the part of the key that carries the position, shared by every head.
 * The expanded form takes each head's own keys and values.
 *
 * Conventions are those of dsaidx.h: caller-owned device memory, nothing
 * allocated or synchronised, every pointer in memory of the current device (the
 * binding refuses others; a pool has no handle that would know), host-side
 * argument errors return before any launch, and what only the device can see (a slot or block id outside the
 * pool, a length beyond its bound) sets the status word, skips the offending
 * key or row and faults nothing.  Status words are sticky: the library never
 * clears them.  Strides are in elements.  A row without a visible key has
 * out 0 and lse -inf.  Sums and softmax statistics are fp32; the weights are
 * rounded to bf16 (2^-8 relative) for the product with the values, so results
 * are off by up to that beside their own rounding.  Waits between a kernel's
 * roles end after 2 s with IDX_ERR_TIMEOUT; the longest one spans the keys one
 * CTA takes of a row (1.3 to 2 us for 64 of them), so a row of tens of millions
 * of keys that is not cut can run into it.
 * Every call may be captured into a CUDA graph.  idx_kernel_timing records the
 * attention calls' kernels too (outside capture).
 */
#ifndef DSAIDX_LATENT_H
#define DSAIDX_LATENT_H

#include "dsaidx.h"

#ifdef __cplusplus
extern "C" {
#endif

#define IDX_LATENT_DIM 512
#define IDX_LATENT_PE_DIM 64
#define IDX_LATENT_RECORD 576            /* elements of one record */
#define IDX_EXPANDED_NOPE_DIM 128
#define IDX_EXPANDED_V_DIM 128
#define IDX_LATENT_MAX_HEADS 1024
#define IDX_ROPE_MAX_DIM 1024
#define IDX_ROPE_MAX_HEADS (1 << 24)

/* Element types of idx_rope. */
typedef enum idx_dtype { IDX_DT_BF16 = 0, IDX_DT_FP16 = 1, IDX_DT_FP32 = 2 } idx_dtype;

/* Scaling of the rotary frequencies for contexts longer than the trained one. */
typedef enum idx_rope_scaling { IDX_ROPE_NONE = 0, IDX_ROPE_LINEAR = 1, IDX_ROPE_YARN = 2 } idx_rope_scaling;

/* Flags of idx_rope and idx_latent_append. */
#define IDX_ROPE_HALF 1u        /* pairs (i, i + rot_dim / 2); default: (2 i, 2 i + 1) */
#define IDX_ROPE_TRANSPOSE 2u   /* the transposed map (the gradient): turns back, amplitude kept (idx_rope only) */

/*
 * Host function: the rotary steps of rot_dim / 2 pairs.  Pair i turns by
 * f_i radians a position, f_i = base^(-2 i / rot_dim); steps_host[i] is
 * f_i / (2 pi) turns as a 64-bit binary fraction, so that position * step
 * modulo 2^64 is the exact fraction of a turn at any position (the error of
 * the angle is that of the double f_i: below 1e-9 radians at 2^20).
 *  LINEAR: f_i / factor.
 *  YARN (Peng et al., "YaRN: Efficient Context Window Extension of Large
 *  Language Models", 2023): f_i (1 - r_i) + f_i / factor * r_i, r_i the ramp
 *  from pair floor(d(beta_fast)) to ceil(d(beta_slow)) with
 *  d(b) = rot_dim ln(original_max_pos / (2 pi b)) / (2 ln base), and the
 *  amplitude 0.1 ln(factor) + 1 (at factor > 1).  The ramp is linear in the pair
 *  index, as models with this scaling are configured and trained; the paper's
 *  text has it linear in original_max_pos / wavelength, which is another ramp
 *  between the same two ends.
 * *amplitude_out (1 unless YARN) scales the turned values.
 * rot_dim even, 2..1024; base > 1; factor >= 1 for LINEAR and YARN.
 */
idx_status idx_rope_steps(int rot_dim, double base, int scaling, double factor, double original_max_pos,
                          double beta_fast, double beta_slow, uint64_t* steps_host, float* amplitude_out);

/*
 * Turns elements [offset, offset + rot_dim) of every head of x [tokens, heads,
 * head_dim] by its token's position and writes y of the same shape (the other
 * elements are copied).  y == x with equal strides turns in place; otherwise
 * x and y must not overlap.  Any strides and alignment (elements of a head
 * are contiguous), but no element is written twice: strides of y at which two
 * heads (in place: their turned parts) share elements, as a broadcast head's
 * stride of 0, are IDX_ERR_INVALID_ARG.  positions_dev: [tokens] int64, any sign.  steps_dev: the
 * rot_dim / 2 steps of idx_rope_steps in device memory.  Angles are exact to
 * about 1e-7 radians; arithmetic in fp32, one rounding to the type.
 * head_dim 1..1024; heads 1..2^24; tokens * heads < 2^33.
 */
idx_status idx_rope(const void* x_dev, int64_t x_token_stride, int64_t x_head_stride, void* y_dev,
                    int64_t y_token_stride, int64_t y_head_stride, int dtype, int64_t tokens, int heads, int head_dim,
                    const int64_t* positions_dev, const uint64_t* steps_dev, int rot_dim, int offset, float amplitude,
                    unsigned flags, void* stream);

/* A caller-owned pool of latent records: num_blocks blocks of block_size
 * records of IDX_LATENT_RECORD bf16 values, contiguous, 128-byte aligned.
 * Slot = block * block_size + offset.  block_size 1..65536, fewer than 2^31
 * slots. */
typedef struct idx_latent_pool {
    void* data_dev;
    int64_t num_blocks;
    int block_size;
} idx_latent_pool;

/*
 * Writes the records of n tokens: latent_dev [n, 512] (row stride
 * latent_stride) is copied, pe_dev [n, 64] (row stride pe_stride) is turned by
 * positions_dev [n] (fp32, one rounding to bf16) or, where steps_dev is null,
 * copied.  slot_mapping_dev [n] int64: a negative slot skips the token; one
 * beyond the pool skips it and sets status_dev (nullable).  Rows 16-byte
 * aligned, strides multiples of 8.  flags: IDX_ROPE_HALF.
 */
idx_status idx_latent_append(const idx_latent_pool* pool, const void* latent_dev, int64_t latent_stride,
                             const void* pe_dev, int64_t pe_stride, const int64_t* positions_dev,
                             const int64_t* slot_mapping_dev, int64_t n, const uint64_t* steps_dev, float amplitude,
                             unsigned flags, int32_t* status_dev, void* stream);

/* Workspace bytes of one absorbed attention call (slots: max_keys = topk;
 * paged: rows = batch, max_keys = max_seq_len), enough for every call of no
 * more rows, heads and keys too, so that one workspace of the largest batch
 * serves the smaller ones.  At most 40 MB.  0 on invalid arguments.  The
 * first word is the call's status (idx_read_device_status); zero the
 * workspace once with idx_workspace_init.  Concurrent calls must not share
 * one. */
size_t idx_latent_workspace_bytes(int64_t rows, int heads, int64_t max_keys);

/*
 * Absorbed attention of every row over the records at its slots.
 *  ql_dev [rows, heads, 512], qp_dev [rows, heads, 64] bf16, 16-byte aligned,
 *  strides positive multiples of 8 (a transposed [heads, rows, 512] is fine).
 *  slots_dev [rows, topk] int64 (row stride slots_stride): the out_slot of the
 *  score calls; negative entries anywhere are skipped, an entry beyond the
 *  pool is skipped and sets the status.  A slot listed twice counts twice.
 *  out_dev [rows, heads, 512] bf16 contiguous, 16-byte aligned; lse_dev nullable [rows, heads] fp32.
 * heads 1..1024, topk 0..2^24, rows * ceil(heads / 64) < 2^31.
 */
idx_status idx_latent_attend_slots(const idx_latent_pool* pool, const void* ql_dev, int64_t ql_row_stride,
                                   int64_t ql_head_stride, const void* qp_dev, int64_t qp_row_stride,
                                   int64_t qp_head_stride, const int64_t* slots_dev, int64_t slots_stride,
                                   int64_t rows, int heads, int topk, float scale, void* out_dev, float* lse_dev,
                                   void* workspace_dev, size_t ws_bytes, void* stream);

/*
 * Absorbed attention of one query a sequence over all its records: logical
 * key s of sequence b is record s % block_size of block
 * block_table_dev[b][s / block_size] (as in idx_score_topk_decode).  A
 * sequence longer than max_seq_len or than its table row, or of negative
 * length, sets the status and gets an empty row; a block id outside the pool
 * sets it and its keys are skipped.  Other arguments as above.
 */
idx_status idx_latent_attend_paged(const idx_latent_pool* pool, const void* ql_dev, int64_t ql_row_stride,
                                   int64_t ql_head_stride, const void* qp_dev, int64_t qp_row_stride,
                                   int64_t qp_head_stride, const int32_t* block_table_dev, int max_blocks_per_seq,
                                   const int32_t* seq_lens_dev, int batch, int max_seq_len, int heads, float scale,
                                   void* out_dev, float* lse_dev, void* workspace_dev, size_t ws_bytes, void* stream);

/*
 * Expanded causal attention of packed prompts:
 *   s = scale * (q[t, h, :128] . kn[j, h] + q[t, h, 128:] . kp[j]),
 *   out[t, h] = sum_j softmax_j(s) v[j, h].
 *  q_dev [total_q, heads, 192], kn_dev and v_dev [total_k, heads, 128],
 *  kp_dev [total_k, 64] (shared by the heads), bf16, 16-byte aligned, strides
 *  multiples of 8 and below 2^31.  cu_seqlens_q_dev / cu_seqlens_k_dev [batch + 1] int32: rows
 *  cu[b]..cu[b+1]-1 belong to sequence b; its queries are its last positions
 *  (query i of n sees keys up to len_k - n + i, none where that is negative).
 *  Keys a query does not see have weight 0, whatever they hold; values of its
 *  own sequence that it does not see have to be finite (0 * inf is NaN).
 *  Offsets that decrease or pass the totals set status_dev (nullable) and the
 *  sequence is skipped (its rows are not written).
 *  out_dev [total_q, heads, 128] bf16 contiguous; lse_dev nullable
 *  [total_q, heads] fp32.  batch <= 4096, total_q, total_k < 2^31.
 */
idx_status idx_latent_attend_expanded(const void* q_dev, int64_t q_row_stride, int64_t q_head_stride,
                                      const void* kn_dev, int64_t kn_row_stride, int64_t kn_head_stride,
                                      const void* kp_dev, int64_t kp_row_stride, const void* v_dev,
                                      int64_t v_row_stride, int64_t v_head_stride, const int32_t* cu_seqlens_q_dev,
                                      const int32_t* cu_seqlens_k_dev, int batch, int64_t total_q, int64_t total_k,
                                      int heads, float scale, void* out_dev, float* lse_dev, int32_t* status_dev,
                                      void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DSAIDX_LATENT_H */
