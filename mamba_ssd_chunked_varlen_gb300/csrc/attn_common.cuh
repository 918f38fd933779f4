// Shared definitions of the paged-cache kernels: the batch and the cache as a
// kernel sees them, and where a token lies.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/ssd_attn.h"

namespace ssd {

// Launches a kernel that begins with pdl_wait() ahead of its predecessor's end, with so
// many bytes of dynamic shared memory.
template <typename... Args>
inline cudaError_t launch_pdl_smem(void (*fn)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                                   Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, args...);
}
template <typename... Args>
inline cudaError_t launch_pdl(void (*fn)(Args...), dim3 grid, int threads, cudaStream_t stream, Args... args)
{
    return launch_pdl_smem(fn, grid, threads, 0, stream, args...);
}

// Smallest row maximum that a quantised row is scaled by: M / a and a / M stay
// normal fp32 numbers for every row, all zeros among them.
constexpr float kKvTiny = 8.673617379884035e-19f;   // 2^-60

constexpr int kKvMaxHeads = 65535;   // kv heads of a call

constexpr float kInt8Max = 127.f;
constexpr float kE4m3Max = 448.f;

// The batch and its cache, passed to kernels by value.
struct KvView {
    void *k, *v;                 // (pages, heads, page, dim)
    float *k_scale, *v_scale;    // (pages, heads, page), null for bf16
    const int32_t *qsl;          // (batch + 1)
    const int32_t *kv_lens;      // (batch)
    const int32_t *table;        // (batch, table_width), rows table_stride apart
    int64_t table_stride, num_pages, total_len;
    uint32_t *errors;            // may be null
    int32_t batch, heads, dim;
    int32_t page, page_shift;    // page = 1 << page_shift
    int32_t table_width, type;
};

__device__ __forceinline__ void kv_error(const KvView &c, uint32_t flag)
{
    if (c.errors)
        atomicOr(c.errors, flag);
}

// Tokens of sequence b in the cache; 0 (and the flag) when its entry is no
// length that the block table can hold.
__device__ __forceinline__ int32_t kv_len_of(const KvView &c, int b)
{
    const int32_t n = c.kv_lens[b];
    if (n < 0 || n > static_cast<int64_t>(c.table_width) << c.page_shift) {
        kv_error(c, SSD_DEVERR_BAD_KV_LEN);
        return 0;
    }
    return n;
}

// The sequence that holds row t, by a whole warp (t the same in every lane):
// the largest b with qsl[b] <= t, found 32 probes at a time; -1 when
// query_start_loc does not place t.
__device__ __forceinline__ int warp_sequence_of(const KvView &c, int64_t t)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, n = c.batch;
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int at = lane * step;
        const bool below = at < n && static_cast<int64_t>(c.qsl[lo + at]) <= t;
        const uint32_t m = __ballot_sync(0xffffffffu, below);
        const int k = m ? 31 - __clz(m) : 0;
        lo += k * step;
        n = min(step, n - k * step);
    }
    return static_cast<int64_t>(c.qsl[lo]) <= t && t < static_cast<int64_t>(c.qsl[lo + 1]) ? lo : -1;
}

// Page and row in the page of token j (0 <= j < kv_len) of sequence b; -1 (and
// the flag) for a page index outside the cache.
__device__ __forceinline__ int64_t kv_page_of(const KvView &c, int b, int32_t j)
{
    const int32_t p = c.table[b * c.table_stride + (j >> c.page_shift)];
    if (p < 0 || p >= c.num_pages) {
        kv_error(c, SSD_DEVERR_BAD_PAGE);
        return -1;
    }
    return p;
}

// Row index (of head_dim elements, or of one scale) in the cache.
__device__ __forceinline__ int64_t kv_row(const KvView &c, int64_t page, int head, int32_t j)
{
    return ((page * c.heads + head) << c.page_shift) + (j & (c.page - 1));
}

// The host-side checks that the three calls share.
ssd_status_t kv_check(KvView *c, const void *k_cache, const void *v_cache, const float *k_scale,
                      const float *v_scale, const int32_t *qsl, const int32_t *kv_lens,
                      const int32_t *block_table, int64_t total_len, int32_t batch,
                      int32_t nheads_kv, int32_t head_dim, int64_t num_pages, int32_t page_size,
                      int32_t table_width, int64_t table_stride, int32_t cache_type,
                      uint32_t *errors);

// A row pitch in elements (0: contiguous): at least the row, a multiple of 16 bytes.
inline bool kv_pitch(int64_t *stride, int64_t row)
{
    if (*stride == 0)
        *stride = row;
    return *stride >= row && *stride % 8 == 0;
}

inline bool kv_aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace ssd
