// Causal grouped-query attention of a ragged batch's new tokens over a paged
// cache: one warp per (row, query head), one pass over the keys with the
// running maximum and sum of the softmax.
#include <cmath>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "attn_common.cuh"

namespace ssd {
namespace {

constexpr int kWarps = 4;

struct AttnParams {
    KvView c;
    __nv_bfloat16 *o;
    const __nv_bfloat16 *q;
    float *lse;
    int64_t o_stride, q_stride;
    int32_t heads, window;
    float scale;
};

__device__ __forceinline__ float cache_value(const KvView &c, const void *base, int64_t i)
{
    if (c.type == SSD_KV_BF16)
        return __bfloat162float(static_cast<const __nv_bfloat16 *>(base)[i]);
    if (c.type == SSD_KV_INT8)
        return static_cast<const int8_t *>(base)[i];
    return __half2float(
        __half(__nv_cvt_fp8_to_halfraw(static_cast<const __nv_fp8_storage_t *>(base)[i], __NV_E4M3)));
}

template <int kDim>
__global__ void __launch_bounds__(kWarps * 32) attn_kernel(AttnParams p)
{
    constexpr int kE = kDim / 32;
    const KvView &c = p.c;
    const int lane = threadIdx.x & 31;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    int bad = 0;
    for (int b = threadIdx.x; b < c.batch; b += kWarps * 32)
        bad |= c.qsl[b + 1] < c.qsl[b] || (b == 0 && c.qsl[0] != 0) ||
               (b == c.batch - 1 && c.qsl[c.batch] != c.total_len);
    if (__syncthreads_or(bad)) {
        kv_error(c, SSD_DEVERR_BAD_QUERY_START_LOC);
        return;
    }
    if (item >= c.total_len * p.heads)
        return;
    const int64_t t = item / p.heads;
    const int h = static_cast<int>(item % p.heads), kvh = h / (p.heads / c.heads);
    const int b = warp_sequence_of(c, t);
    if (b < 0)
        return;
    const int64_t at = kv_len_of(c, b) - static_cast<int64_t>(c.qsl[b + 1]) + t;
    const int64_t lo = p.window > 0 && at - p.window + 1 > 0 ? at - p.window + 1 : 0;
    float q[kE], o[kE], m = -INFINITY, l = 0.f;
    for (int e = 0; e < kE; ++e) {
        q[e] = __bfloat162float(p.q[t * p.q_stride + h * kDim + e * 32 + lane]);
        o[e] = 0.f;
    }
    for (int64_t j = lo; j <= at; ++j) {
        const int64_t page = kv_page_of(c, b, static_cast<int32_t>(j));
        if (page < 0)
            continue;
        const int64_t row = kv_row(c, page, kvh, static_cast<int32_t>(j));
        float s = 0.f;
        for (int e = 0; e < kE; ++e)
            s += q[e] * cache_value(c, c.k, row * kDim + e * 32 + lane);
        for (int w = 16; w; w >>= 1)
            s += __shfl_xor_sync(0xffffffffu, s, w);
        s *= p.scale * (c.k_scale ? c.k_scale[row] : 1.f);
        const float mn = fmaxf(m, s);
        const float a = m == -INFINITY ? 0.f : expf(m - mn), w = expf(s - mn);
        l = l * a + w;
        const float wv = w * (c.v_scale ? c.v_scale[row] : 1.f);
        for (int e = 0; e < kE; ++e)
            o[e] = o[e] * a + wv * cache_value(c, c.v, row * kDim + e * 32 + lane);
        m = mn;
    }
    for (int e = 0; e < kE; ++e)
        p.o[t * p.o_stride + h * kDim + e * 32 + lane] =
            __float2bfloat16_rn(m == -INFINITY ? 0.f : o[e] / l);
    if (p.lse && lane == 0)
        p.lse[item] = m == -INFINITY ? -INFINITY : m + logf(l);
}

}  // namespace
}  // namespace ssd

extern "C" {

size_t ssd_attn_varlen_workspace_size(int64_t total_len, int32_t batch, int32_t nheads,
                                      int32_t nheads_kv, int32_t head_dim)
{
    if (total_len < 0 || total_len > INT32_MAX / 2 || batch < 0 || nheads <= 0 || nheads_kv <= 0 || nheads % nheads_kv != 0 ||
        nheads / nheads_kv > 128 || (head_dim != 64 && head_dim != 128))
        return 0;
    return 256;
}

ssd_status_t ssd_attn_varlen_fwd(void *o, float *lse, const void *q, const void *k_cache,
                                 const void *v_cache, const float *k_scale, const float *v_scale,
                                 const int32_t *query_start_loc, const int32_t *kv_lens,
                                 const int32_t *block_table, int64_t total_len, int32_t batch,
                                 int32_t nheads, int32_t nheads_kv, int32_t head_dim,
                                 int64_t num_pages, int32_t page_size, int32_t table_width,
                                 int64_t table_stride, int32_t cache_type, int64_t o_stride,
                                 int64_t q_stride, float softmax_scale, int32_t window,
                                 void *workspace, size_t workspace_bytes, uint32_t *errors,
                                 ssd_stream_t stream_)
{
    using namespace ssd;
    AttnParams p;
    const ssd_status_t st =
        kv_check(&p.c, k_cache, v_cache, k_scale, v_scale, query_start_loc, kv_lens, block_table,
                 total_len, batch, nheads_kv, head_dim, num_pages, page_size, table_width,
                 table_stride, cache_type, errors);
    if (st != SSD_OK)
        return st;
    if (nheads <= 0 || nheads % nheads_kv != 0 || window < 0 || !std::isfinite(softmax_scale))
        return SSD_ERR_INVALID_ARG;
    if (nheads / nheads_kv > 128)
        return SSD_ERR_UNSUPPORTED;
    const int64_t row = static_cast<int64_t>(nheads) * head_dim;
    if (!kv_pitch(&o_stride, row) || !kv_pitch(&q_stride, row))
        return SSD_ERR_INVALID_ARG;
    if (total_len == 0)
        return SSD_OK;
    if (batch == 0 || !o || !q || !kv_aligned16(o) || !kv_aligned16(q))
        return SSD_ERR_INVALID_ARG;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
        workspace_bytes < ssd_attn_varlen_workspace_size(total_len, batch, nheads, nheads_kv, head_dim))
        return SSD_ERR_WORKSPACE;
    p.o = static_cast<__nv_bfloat16 *>(o);
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.lse = lse;
    p.o_stride = o_stride;
    p.q_stride = q_stride;
    p.heads = nheads;
    p.window = window;
    p.scale = softmax_scale;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    const unsigned grid = static_cast<unsigned>((total_len * nheads + kWarps - 1) / kWarps);
    if (head_dim == 128)
        attn_kernel<128><<<grid, kWarps * 32, 0, stream>>>(p);
    else
        attn_kernel<64><<<grid, kWarps * 32, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
