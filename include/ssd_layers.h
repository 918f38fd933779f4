/*
 * ssd_layers.h -- C ABI of the operators around the scan (ssd_scan.h) and the
 * attention (ssd_attn.h) in a hybrid model's layers: the short causal
 * convolution before a scan, the selective scan whose step and decay are each
 * channel's own, the root-mean-square norm, and rotary positions.
 *
 * They take the ragged batch of those two:
 *
 *   query_start_loc   int32 (batch + 1): the new tokens of sequence b are rows
 *                     [qsl[b], qsl[b+1]) of the token-major tensors.  qsl[0] is
 *                     0; qsl[batch] may be less than total_len (a padded batch):
 *                     rows behind the last sequence are neither used nor written
 *   has_initial_state uint8 (batch) or NULL (all false); nonzero = true
 *   cache_indices     uint32 (batch): pool slot of sequence b.  SSD_NO_SLOT is
 *                     none: the state starts at zero and is not kept.  Other
 *                     sequences' slots must be distinct
 *
 * Only the pool slots that cache_indices names are written, each with the state
 * after its sequence's last token, also for a sequence of length 0 (its initial
 * state, or zeros).
 *
 * Token-major tensors have rows a stride of their own apart, in elements
 * (0: contiguous), at least the row and a multiple of 8; they are 16-byte aligned.
 * Outputs must not overlap inputs where it is not said that they may.
 *
 * Conventions are those of ssd_scan.h: device pointers owned by the caller,
 * asynchronous on `stream`, SSD_OK or a status with nothing launched.  Errors
 * that only the device can see are OR-ed into `errors` (device memory, or NULL),
 * which the library never clears:
 *
 *   SSD_DEVERR_BAD_QUERY_START_LOC  qsl[0] != 0, decreasing, or above total_len: a
 *                     sequence with such a bound is skipped, the rows that no good
 *                     sequence holds and the skipped sequences' slots are
 *                     unspecified; where offsets decrease, all rows and all named slots
 *                     are (no other memory is touched)
 *   SSD_DEVERR_BAD_CACHE_INDEX      cache_indices[b] >= max_slots and not
 *                     SSD_NO_SLOT: taken for SSD_NO_SLOT
 */
#ifndef SSD_LAYERS_H_
#define SSD_LAYERS_H_

#include "ssd_attn.h"
#include "ssd_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SSD_NO_SLOT 0xffffffffu

/* The short causal convolution of every channel, for prompts and single tokens:
 *
 *   y[t,c] = act(bias[c] + sum_{j < width} weight[c,j] u[t - (width-1) + j, c])
 *
 * with u = x in the sequence and, before its first token, the last inputs that
 * its slot holds (zeros without has_initial_state); act is silu, v / (1 + e^-v),
 * or nothing.  The slot gets the last width - 1 inputs.  (Here and below, silu of v < -87,
 * smaller than 2e-36, is taken for 0.)
 *
 *   y, x       bf16 (total_len, channels), rows y_stride and x_stride apart, e.g.
 *              column slices of a fused projection
 *   weight     fp32 (channels, width);  bias fp32 (channels) or NULL (zeros)
 *   conv_pool  bf16 (max_slots, width - 1, channels): the oldest input first
 *
 * Supported: width 2, 3 or 4; channels a multiple of 8, at most 2^20.  Sums are
 * fp32, y is rounded once. */
SSD_API ssd_status_t ssd_causal_conv_varlen_fwd(
    void *y, const void *x, const float *weight, const float *bias, void *conv_pool,
    const int32_t *query_start_loc, const uint8_t *has_initial_state,
    const uint32_t *cache_indices, int64_t total_len, int32_t batch, int32_t channels,
    int32_t width, int64_t max_slots, int64_t y_stride, int64_t x_stride, int32_t silu,
    uint32_t *errors, ssd_stream_t stream);

/* The selective scan whose step and decay are each channel's own, for prompts and single
 * tokens.  For every channel c and state n:
 *
 *   d_t = softplus(dt[t,c] + dt_bias[c])      (plain dt + dt_bias when dt_softplus == 0)
 *   h_n = exp(d_t A[c,n]) h_n + d_t x[t,c] B[t,n]
 *   y[t,c] = (sum_n C[t,n] h_n + D[c] x[t,c]) silu(z[t,c])
 *
 * from the slot's states, or zeros, at each sequence's start (the scan of ssd_scan.h has
 * one step and decay per head).
 *
 *   y, x, dt, z  bf16 (total_len, channels);  z NULL: no gate
 *   B, C         bf16 (total_len, dstate)
 *   A            fp32 (channels, dstate);  D, dt_bias fp32 (channels) or NULL (zeros)
 *   ssm_pool     (max_slots, channels, dstate), fp32, or bf16: widened when read, rounded
 *                when written (pool_type)
 *   strides      of the token-major tensors, or NULL: all contiguous
 *   workspace    at least ssd_selective_scan_varlen_workspace_size bytes, 256-byte aligned;
 *                needs no initialisation; one call at a time per workspace
 *
 * A call of exactly as many rows as sequences (total_len == batch) is taken for a step of single
 * tokens: a longer sequence in it is right, but waits for memory at every token.  Batches padded
 * with empty sequences that may hold prompts do better with any other number of rows.
 *
 * Supported: dstate 8, 16, 32 or 64; channels a multiple of 8, at most 2^20; strides below
 * 2^31.  States and sums are fp32, y is rounded once. */
typedef enum {
    SSD_POOL_FP32 = 0,
    SSD_POOL_BF16 = 1
} ssd_pool_type_t;

typedef struct {
    int64_t y, x, dt, B, C, z;   /* elements between consecutive tokens; 0: contiguous */
} ssd_selective_strides_t;

/* Bytes of device scratch that the call needs for these sizes, and enough for every call
 * that is not larger in any of them; 0 when they are invalid or unsupported. */
SSD_API size_t ssd_selective_scan_varlen_workspace_size(int64_t total_len, int32_t batch,
                                                        int32_t channels, int32_t dstate);

SSD_API ssd_status_t ssd_selective_scan_varlen_fwd(
    void *y, const void *x, const void *dt, const float *A, const void *B, const void *C,
    const float *D, const void *z, const float *dt_bias, void *ssm_pool,
    const int32_t *query_start_loc, const uint8_t *has_initial_state,
    const uint32_t *cache_indices, int64_t total_len, int32_t batch, int32_t channels,
    int32_t dstate, int64_t max_slots, int32_t pool_type, int32_t dt_softplus,
    const ssd_selective_strides_t *strides, void *workspace, size_t workspace_bytes,
    uint32_t *errors, ssd_stream_t stream);

/* Root-mean-square norm over groups of dim / ngroups columns.  For each row and group
 *
 *   y = s weight / sqrt(mean s^2 + eps)
 *
 * with s = x, or x + residual, which is written back to residual (rounded to
 * bf16; the norm is that of the sum before), or x silu(gate).
 *
 *   x          bf16 (rows, dim);  gate, residual likewise or NULL, not both
 *   weight     fp32 (dim) or NULL (ones)
 *   y          (rows, dim) in bf16, or in 8-bit codes (out_type, ssd_kv_type_t); in
 *              bf16 it may be x or gate itself
 *   scale      fp32 (rows, ngroups) with 8-bit codes, else NULL: an element stands
 *              for code * scale.  Codes and scales are those that ssd_attn.h defines
 *              for cache rows, of each row's groups: a group with an infinity or a
 *              NaN gets codes 0 and scale NaN
 *
 * Rows are any multiple of 8 elements apart that is not below dim.  Supported: dim /
 * ngroups a multiple of 8, at most 32,768; eps from 2^-80 to 1.  s, and with codes s
 * weight, has to stay in fp32's range (the square need not).  All in fp32, rounded once. */
SSD_API ssd_status_t ssd_rms_norm_fwd(
    void *y, float *scale, const void *x, void *residual, const void *gate, const float *weight,
    int64_t rows, int32_t dim, int32_t ngroups, int32_t out_type, float eps, int64_t y_stride,
    int64_t x_stride, int64_t residual_stride, int64_t gate_stride, ssd_stream_t stream);

/* Rotary positions.  The first rotary_dim elements of a head are pairs (a, b), element
 * i with rotary_dim / 2 + i, or neighbours 2 i and 2 i + 1 (interleaved); pair i of
 * the token at position p becomes
 *
 *   a' = magnitude (a cos(p f_i) - b sin(p f_i)),  b' = magnitude (b cos(p f_i) + a sin(p f_i))
 *
 * and the rest of the head stays.  Frequencies are a table of turns: f_i / (2 pi)
 * as a 64-bit binary fraction, so that p f_i modulo a turn is one integer product,
 * exact at any position; ssd_rope_table makes it.  Scaled frequencies (for contexts
 * longer than a model was trained on) are other values of f_i and magnitude.
 *
 *   turns      uint64 (rotary_dim / 2), device memory
 *   kv_lens    int32 (batch), as in ssd_attn.h: row t of sequence b is its token
 *              kv_lens[b] - qsl[b+1] + t.  Rows at a negative position are padding:
 *              neither used nor written, like rows that no sequence holds
 *
 * Supported: rotary_dim a multiple of 16, at most head_dim; head_dim 64 or 128. */

/* Host only: turns[i] = frequencies[i] / (2 pi) 2^64, rounded, for n frequencies in
 * radians per position, each at least 0 and below 2 pi (else SSD_ERR_INVALID_ARG). */
SSD_API ssd_status_t ssd_rope_table(uint64_t *turns, const double *frequencies, int32_t n);

/* Rotates the new tokens' queries and keys, or one of them (the other's pointers
 * NULL): q and q_out bf16 (total_len, nheads, head_dim), k and k_out bf16 (total_len,
 * nheads_kv, head_dim).  An output may be its input, at the same stride.  The cosine,
 * the sine and the products are fp32, outputs are rounded once. */
SSD_API ssd_status_t ssd_rope_varlen_fwd(
    void *q_out, const void *q, void *k_out, const void *k, const uint64_t *turns,
    const int32_t *query_start_loc, const int32_t *kv_lens, int64_t total_len, int32_t batch,
    int32_t nheads, int32_t nheads_kv, int32_t head_dim, int32_t rotary_dim, int32_t interleaved,
    float magnitude, int64_t q_out_stride, int64_t q_stride, int64_t k_out_stride,
    int64_t k_stride, uint32_t *errors, ssd_stream_t stream);

/* ssd_rope_varlen_fwd of q and k and ssd_kv_cache_write of the rotated k and of v in
 * one launch: what the attention needs of a projection's output.  The rotated k is
 * quantised from fp32.  Arguments as for these two; query_start_loc as above. */
SSD_API ssd_status_t ssd_rope_kv_cache_write(
    void *q_out, const void *q, const void *k, const void *v, const uint64_t *turns,
    void *k_cache, void *v_cache, float *k_scale, float *v_scale, const int32_t *query_start_loc,
    const int32_t *kv_lens, const int32_t *block_table, int64_t total_len, int32_t batch,
    int32_t nheads, int32_t nheads_kv, int32_t head_dim, int32_t rotary_dim, int32_t interleaved,
    float magnitude, int64_t num_pages, int32_t page_size, int32_t table_width,
    int64_t table_stride, int32_t cache_type, int64_t q_out_stride, int64_t q_stride,
    int64_t k_stride, int64_t v_stride, uint32_t *errors, ssd_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SSD_LAYERS_H_ */
