/*
 * ssd_attn.h -- C ABI of the paged key/value cache and the attention over it.
 *
 * These operators serve the attention layers of a hybrid model, whose scan
 * layers use ssd_scan.h, on the same ragged batch: query_start_loc names the
 * new tokens of every sequence, as it does for the scan.
 *
 * One description of the batch serves all three calls:
 *
 *   query_start_loc int32 (batch + 1): the new tokens of sequence b are rows
 *                   [qsl[b], qsl[b+1]) of the token-major tensors
 *   kv_lens         int32 (batch): tokens of sequence b in the cache, the new
 *                   ones counted; its new tokens are its last ones, so row t
 *                   is its token kv_lens[b] - qsl[b+1] + t.  Rows at a
 *                   negative position (a padded batch, kv_lens[b] smaller than
 *                   the sequence's rows) are padding: not written, read back
 *                   as zeros, their attention is zero
 *   block_table     int32 (batch, table_width), rows table_stride elements
 *                   apart: token j of sequence b lies in row j % page_size of
 *                   page block_table[b][j / page_size]; entries past the
 *                   sequence's last page are not read
 *
 * The cache:
 *
 *   k_cache, v_cache (num_pages, nheads_kv, page_size, head_dim), bf16, or
 *                   8-bit codes (cache_type)
 *   k_scale, v_scale fp32 (num_pages, nheads_kv, page_size) with 8-bit codes,
 *                   else NULL: an element stands for code * scale
 *
 * A row x (head_dim elements of one token and head) is quantised as it is
 * written, all in fp32: a = max(max|x|, 2^-60), code = round(x * (M / a)),
 * scale = a / M, with M = 127 (int8, ties to even) or 448 (fp8 e4m3, its own
 * rounding to nearest even).  A row that holds an infinity or a NaN gets codes
 * 0 and scale NaN: it reads back as NaN, and so is every attention row that
 * sees it, and no other.  A cache filled in another way may have scales of any
 * finite value, or NaN; e4m3's NaN codes may lie only in rows that no sequence
 * holds.
 *
 * Conventions are those of ssd_scan.h: device pointers owned by the caller,
 * asynchronous on `stream`, SSD_OK or a status with nothing launched.  Errors
 * that only the device can see are OR-ed into `errors` (device memory, or
 * NULL): the library never clears that word, so one word may collect the flags
 * of a whole step.
 */
#ifndef SSD_ATTN_H_
#define SSD_ATTN_H_

#include "ssd_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SSD_KV_BF16 = 0,
    SSD_KV_FP8_E4M3 = 1,
    SSD_KV_INT8 = 2
} ssd_kv_type_t;

/* Device-side error flags beside those of ssd_scan.h.
 * SSD_DEVERR_BAD_QUERY_START_LOC: cache calls skip the rows that no sequence
 * holds (a read zeroes them); attention computes and writes nothing. */
#define SSD_DEVERR_BAD_KV_LEN 0x8u  /* kv_lens[b] < 0 or more than table_width pages hold: the
                                       sequence counts as having no token in the cache */
#define SSD_DEVERR_BAD_PAGE   0x10u /* a page index outside [0, num_pages): not written; its
                                       keys and values read as zeros */

/* Writes the new tokens' keys and values into the cache.
 *
 *   k, v       bf16 (total_len, nheads_kv, head_dim), rows k_stride and
 *              v_stride elements apart (0: contiguous), e.g. column slices of
 *              a fused projection; strides multiples of 8, 16-byte aligned
 *
 * Supported: head_dim 64 or 128; page_size 16, 32, 64, 128 or 256; at most
 * 65,535 kv heads.  Cache pointers 16-byte aligned.  Two rows of one call must
 * not share a cache row. */
SSD_API ssd_status_t ssd_kv_cache_write(
    const void *k, const void *v, void *k_cache, void *v_cache, float *k_scale, float *v_scale,
    const int32_t *query_start_loc, const int32_t *kv_lens, const int32_t *block_table,
    int64_t total_len, int32_t batch, int32_t nheads_kv, int32_t head_dim, int64_t num_pages,
    int32_t page_size, int32_t table_width, int64_t table_stride, int32_t cache_type,
    int64_t k_stride, int64_t v_stride, uint32_t *errors, ssd_stream_t stream);

/* Reads rows back: row t of k and v (bf16, as above) gets the cache's values
 * of the token that ssd_kv_cache_write would write from it, code * scale in
 * fp32 rounded once to bf16.  With query_start_loc the running sum of kv_lens
 * it reads whole contexts. */
SSD_API ssd_status_t ssd_kv_cache_read(
    void *k, void *v, const void *k_cache, const void *v_cache, const float *k_scale,
    const float *v_scale, const int32_t *query_start_loc, const int32_t *kv_lens,
    const int32_t *block_table, int64_t total_len, int32_t batch, int32_t nheads_kv,
    int32_t head_dim, int64_t num_pages, int32_t page_size, int32_t table_width,
    int64_t table_stride, int32_t cache_type, int64_t k_stride, int64_t v_stride,
    uint32_t *errors, ssd_stream_t stream);

/* Bytes of device scratch that ssd_attn_varlen_fwd needs for these sizes, and
 * enough for every call that is not larger in any of them (fewer kv heads, as in
 * another layer, among them), whatever the contexts' lengths; or 0 when they are
 * invalid or unsupported. */
SSD_API size_t ssd_attn_varlen_workspace_size(int64_t total_len, int32_t batch, int32_t nheads,
                                              int32_t nheads_kv, int32_t head_dim);

/* Causal grouped-query attention of the new tokens over the cache, which
 * already holds them.  For query head h, kv head h / (nheads / nheads_kv) and
 * the query at position i of its sequence:
 *
 *   S_j = softmax_scale * q_i . k_j   for i - window < j <= i (all j <= i with window 0)
 *   o_i = sum_j exp(S_j) v_j / sum_j exp(S_j),   lse_i = ln sum_j exp(S_j)
 *
 * A row that sees no key gets o = 0 and lse = -infinity.  Keys that the mask hides
 * do not count, whatever they hold.  Over a bf16 cache an infinity in V is the
 * result of the rows that see it (where its probability is too small for fp32
 * it may be NaN), and NaN is NaN.  Probabilities are relative to a reference that
 * may lag behind the maximum (by 2^16 at most), so that sums of p v pass through
 * numbers larger than the result: values up to 2^80 in magnitude are safe at any
 * length, larger ones may give infinities.
 *
 *   o, q       bf16 (total_len, nheads, head_dim), rows o_stride and q_stride
 *              elements apart (0: contiguous; multiples of 8); 16-byte aligned
 *   lse        fp32 (total_len, nheads) or NULL
 *   workspace  at least ssd_attn_varlen_workspace_size bytes, 256-byte aligned;
 *              needs no initialisation; one call at a time per workspace
 *
 * Sums and softmax statistics are fp32; probabilities (times v's scale) enter the
 * product with v as one bf16 each, or as two where a sequence has at most 16 query
 * rows a kv head.  Supported as above, nheads a multiple of nheads_kv, at most 128
 * query heads a kv head; window >= 0 (one that no context can pass is none);
 * softmax_scale finite, and so is its product with log2(e). */
SSD_API ssd_status_t ssd_attn_varlen_fwd(
    void *o, float *lse, const void *q, const void *k_cache, const void *v_cache,
    const float *k_scale, const float *v_scale, const int32_t *query_start_loc,
    const int32_t *kv_lens, const int32_t *block_table, int64_t total_len, int32_t batch,
    int32_t nheads, int32_t nheads_kv, int32_t head_dim, int64_t num_pages, int32_t page_size,
    int32_t table_width, int64_t table_stride, int32_t cache_type, int64_t o_stride,
    int64_t q_stride, float softmax_scale, int32_t window, void *workspace,
    size_t workspace_bytes, uint32_t *errors, ssd_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SSD_ATTN_H_ */
