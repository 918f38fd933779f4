// Paged key/value cache: rows quantised as they are written, and read back.
//
// Write, per row x of head_dim elements (one token, one head, K or V):
//     a = max(max|x|, 2^-60),  code = round(x * (M / a)),  scale = a / M
// Read: x' = bf16(code * scale).  One pass over the rows in each direction.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "attn_common.cuh"

namespace ssd {

ssd_status_t kv_check(KvView *c, const void *k_cache, const void *v_cache, const float *k_scale,
                      const float *v_scale, const int32_t *qsl, const int32_t *kv_lens,
                      const int32_t *block_table, int64_t total_len, int32_t batch,
                      int32_t nheads_kv, int32_t head_dim, int64_t num_pages, int32_t page_size,
                      int32_t table_width, int64_t table_stride, int32_t cache_type,
                      uint32_t *errors)
{
    if (total_len < 0 || batch < 0 || nheads_kv <= 0 || head_dim <= 0 || num_pages <= 0 ||
        page_size <= 0 || table_width < 0)
        return SSD_ERR_INVALID_ARG;
    if (cache_type != SSD_KV_BF16 && cache_type != SSD_KV_FP8_E4M3 && cache_type != SSD_KV_INT8)
        return SSD_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128)
        return SSD_ERR_UNSUPPORTED;
    if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128 &&
        page_size != 256)
        return SSD_ERR_UNSUPPORTED;
    if (table_stride == 0)
        table_stride = table_width;
    if (table_stride < table_width)
        return SSD_ERR_INVALID_ARG;
    if (total_len > INT32_MAX / 2 || batch > INT32_MAX / 2 || num_pages > INT32_MAX / 2 / nheads_kv ||
        static_cast<int64_t>(table_width) * page_size > INT32_MAX / 2 || nheads_kv > 65535)
        return SSD_ERR_UNSUPPORTED;
    if (total_len > 0 && batch > 0) {
        if (!qsl || !kv_lens || (table_width > 0 && !block_table))
            return SSD_ERR_INVALID_ARG;
        if (!k_cache || !v_cache)
            return SSD_ERR_INVALID_ARG;
        if (cache_type != SSD_KV_BF16 && (!k_scale || !v_scale))
            return SSD_ERR_INVALID_ARG;
    }
    if (!kv_aligned16(k_cache) || !kv_aligned16(v_cache) || !kv_aligned16(k_scale) ||
        !kv_aligned16(v_scale))
        return SSD_ERR_INVALID_ARG;
    c->k = const_cast<void *>(k_cache);
    c->v = const_cast<void *>(v_cache);
    c->k_scale = const_cast<float *>(k_scale);
    c->v_scale = const_cast<float *>(v_scale);
    c->qsl = qsl;
    c->kv_lens = kv_lens;
    c->table = block_table;
    c->table_stride = table_stride;
    c->num_pages = num_pages;
    c->total_len = total_len;
    c->errors = errors;
    c->batch = batch;
    c->heads = nheads_kv;
    c->dim = head_dim;
    c->page = page_size;
    c->page_shift = 0;
    while ((1 << c->page_shift) < page_size)
        ++c->page_shift;
    c->table_width = table_width;
    c->type = cache_type;
    return SSD_OK;
}

namespace {

constexpr int kWarps = 8;          // warps of a CTA
constexpr int kRowsPerLane = 4;    // rows that a lane has in flight

// Eight bf16 values of a row as fp32.
__device__ __forceinline__ void widen8(const uint4 &r, float (&x)[8])
{
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b)
{
    const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&t);
}

template <int kType>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv)
{
    uint32_t w[2] = {0u, 0u};
    if constexpr (kType == SSD_KV_INT8) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i >> 2] |= (static_cast<uint32_t>(__float2int_rn(__fmul_rn(x[i], inv))) & 0xffu)
                         << (8 * (i & 3));
    } else {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const uint32_t p = __nv_cvt_float2_to_fp8x2(
                make_float2(__fmul_rn(x[i], inv), __fmul_rn(x[i + 1], inv)), __NV_SATFINITE,
                __NV_E4M3);
            w[i >> 2] |= p << (8 * (i & 3));
        }
    }
    return make_uint2(w[0], w[1]);
}

template <int kType>
__device__ __forceinline__ void decode8(const uint2 &r, float (&x)[8])
{
    const uint32_t w[2] = {r.x, r.y};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t b = (w[i >> 2] >> (8 * (i & 3))) & 0xffu;
        if constexpr (kType == SSD_KV_INT8)
            x[i] = static_cast<float>(static_cast<int8_t>(b));
        else
            x[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(b),
                                                               __NV_E4M3)));
    }
}

// One warp: row t's K and V rows [first, first + 4 * 256 / dim) of the token's
// 2 * heads.  A row is dim / 8 lanes of eight elements.
template <int kType, int kDim, bool kWrite>
__global__ void __launch_bounds__(kWarps * 32)
    kv_copy_kernel(KvView c, __nv_bfloat16 *k, __nv_bfloat16 *v, int64_t k_stride, int64_t v_stride)
{
    constexpr int kLanes = kDim / 8;           // lanes of a row
    constexpr int kAtOnce = 32 / kLanes;       // rows of the warp's one load
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    if (blockIdx.x == 0 && blockIdx.y == 0) {   // one CTA looks the offsets over
        bool bad = false;
        for (int b = threadIdx.x; b < c.batch; b += kWarps * 32)
            bad = bad || c.qsl[b + 1] < c.qsl[b] || (b == 0 && c.qsl[0] != 0) ||
                  (b == c.batch - 1 && c.qsl[c.batch] != c.total_len);
        if (bad)
            kv_error(c, SSD_DEVERR_BAD_QUERY_START_LOC);
    }
    if (t >= c.total_len)
        return;
    const int first = blockIdx.y * (kAtOnce * kRowsPerLane);
    const int sub = lane / kLanes, col = (lane % kLanes) * 8;
    const int rows = 2 * c.heads;
    uint4 raw[kRowsPerLane];
    if constexpr (kWrite) {
        // the rows do not depend on where they go: their loads start first
#pragma unroll
        for (int i = 0; i < kRowsPerLane; ++i) {
            const int r = first + i * kAtOnce + sub;
            if (r < rows) {
                const bool is_v = r >= c.heads;
                const __nv_bfloat16 *src = is_v ? v + t * v_stride + (r - c.heads) * kDim
                                                : k + t * k_stride + r * kDim;
                raw[i] = *reinterpret_cast<const uint4 *>(src + col);
            }
        }
    }
    const int b = warp_sequence_of(c, t);
    const int32_t len = b < 0 ? 0 : kv_len_of(c, b);
    const int64_t j = b < 0 ? -1 : len - static_cast<int64_t>(c.qsl[b + 1]) + t;
    const int64_t page = j < 0 ? -1 : kv_page_of(c, b, static_cast<int32_t>(j));
    if (kWrite && page < 0)
        return;
#pragma unroll
    for (int i = 0; i < kRowsPerLane; ++i) {
        const int r = first + i * kAtOnce + sub;
        const bool mine = r < rows;
        const bool is_v = r >= c.heads;
        const int head = is_v ? r - c.heads : r;
        const int64_t row = kv_row(c, page, head, static_cast<int32_t>(j));
        if constexpr (kWrite) {
            if constexpr (kType == SSD_KV_BF16) {
                if (mine)
                    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(is_v ? c.v : c.k) +
                                               row * kDim + col) = raw[i];
            } else {
                constexpr float kTop = kType == SSD_KV_INT8 ? kInt8Max : kE4m3Max;
                float x[8];
                widen8(mine ? raw[i] : make_uint4(0, 0, 0, 0), x);
                float a = 0.f;
                bool finite = true;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    a = fmaxf(a, fabsf(x[e]));
                    finite = finite && fabsf(x[e]) <= 3.4e38f;
                }
                uint32_t bad = finite ? 0u : 1u;
#pragma unroll
                for (int o = 1; o < kLanes; o <<= 1) {
                    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
                    bad |= __shfl_xor_sync(0xffffffffu, bad, o);
                }
                a = fmaxf(a, kKvTiny);
                if (mine) {
                    const uint2 w = bad ? make_uint2(0, 0) : encode8<kType>(x, __fdiv_rn(kTop, a));
                    *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(is_v ? c.v : c.k) +
                                               row * kDim + col) = w;
                    if (col == 0)
                        (is_v ? c.v_scale : c.k_scale)[row] =
                            bad ? __int_as_float(0x7fffffff) : __fdiv_rn(a, kTop);
                }
            }
        } else if (mine) {
            uint4 out = make_uint4(0, 0, 0, 0);
            if (page >= 0) {
                if constexpr (kType == SSD_KV_BF16) {
                    out = *reinterpret_cast<const uint4 *>(
                        static_cast<const __nv_bfloat16 *>(is_v ? c.v : c.k) + row * kDim + col);
                } else {
                    const float s = (is_v ? c.v_scale : c.k_scale)[row];
                    float x[8];
                    decode8<kType>(*reinterpret_cast<const uint2 *>(
                                       static_cast<const uint8_t *>(is_v ? c.v : c.k) + row * kDim + col),
                                   x);
                    out = make_uint4(bf16_pair(x[0] * s, x[1] * s), bf16_pair(x[2] * s, x[3] * s),
                                     bf16_pair(x[4] * s, x[5] * s), bf16_pair(x[6] * s, x[7] * s));
                }
            }
            __nv_bfloat16 *dst = is_v ? v + t * v_stride + head * kDim : k + t * k_stride + head * kDim;
            *reinterpret_cast<uint4 *>(dst + col) = out;
        }
    }
}

template <int kType, int kDim, bool kWrite>
cudaError_t launch(const KvView &c, void *k, void *v, int64_t ks, int64_t vs, cudaStream_t stream)
{
    constexpr int kRows = 32 / (kDim / 8) * kRowsPerLane;
    const dim3 grid(static_cast<unsigned>((c.total_len + kWarps - 1) / kWarps),
                    (2 * c.heads + kRows - 1) / kRows);
    kv_copy_kernel<kType, kDim, kWrite><<<grid, kWarps * 32, 0, stream>>>(
        c, static_cast<__nv_bfloat16 *>(k), static_cast<__nv_bfloat16 *>(v), ks, vs);
    return cudaGetLastError();
}

template <bool kWrite>
ssd_status_t copy(KvView &c, void *k, void *v, int64_t ks, int64_t vs, ssd_stream_t stream_)
{
    const int64_t row = static_cast<int64_t>(c.heads) * c.dim;
    if (!kv_pitch(&ks, row) || !kv_pitch(&vs, row))
        return SSD_ERR_INVALID_ARG;
    if (c.total_len == 0)
        return SSD_OK;
    if (c.batch == 0)   // rows that no sequence holds
        return SSD_ERR_INVALID_ARG;
    if (!k || !v || !kv_aligned16(k) || !kv_aligned16(v))
        return SSD_ERR_INVALID_ARG;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    cudaError_t e;
    const bool wide = c.dim == 128;
    if (c.type == SSD_KV_BF16)
        e = wide ? launch<SSD_KV_BF16, 128, kWrite>(c, k, v, ks, vs, stream)
                 : launch<SSD_KV_BF16, 64, kWrite>(c, k, v, ks, vs, stream);
    else if (c.type == SSD_KV_INT8)
        e = wide ? launch<SSD_KV_INT8, 128, kWrite>(c, k, v, ks, vs, stream)
                 : launch<SSD_KV_INT8, 64, kWrite>(c, k, v, ks, vs, stream);
    else
        e = wide ? launch<SSD_KV_FP8_E4M3, 128, kWrite>(c, k, v, ks, vs, stream)
                 : launch<SSD_KV_FP8_E4M3, 64, kWrite>(c, k, v, ks, vs, stream);
    return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // namespace
}  // namespace ssd

extern "C" {

ssd_status_t ssd_kv_cache_write(const void *k, const void *v, void *k_cache, void *v_cache,
                                float *k_scale, float *v_scale, const int32_t *query_start_loc,
                                const int32_t *kv_lens, const int32_t *block_table,
                                int64_t total_len, int32_t batch, int32_t nheads_kv,
                                int32_t head_dim, int64_t num_pages, int32_t page_size,
                                int32_t table_width, int64_t table_stride, int32_t cache_type,
                                int64_t k_stride, int64_t v_stride, uint32_t *errors,
                                ssd_stream_t stream)
{
    ssd::KvView c;
    const ssd_status_t st = ssd::kv_check(&c, k_cache, v_cache, k_scale, v_scale, query_start_loc,
                                          kv_lens, block_table, total_len, batch, nheads_kv,
                                          head_dim, num_pages, page_size, table_width,
                                          table_stride, cache_type, errors);
    if (st != SSD_OK)
        return st;
    return ssd::copy<true>(c, const_cast<void *>(k), const_cast<void *>(v), k_stride, v_stride,
                           stream);
}

ssd_status_t ssd_kv_cache_read(void *k, void *v, const void *k_cache, const void *v_cache,
                               const float *k_scale, const float *v_scale,
                               const int32_t *query_start_loc, const int32_t *kv_lens,
                               const int32_t *block_table, int64_t total_len, int32_t batch,
                               int32_t nheads_kv, int32_t head_dim, int64_t num_pages,
                               int32_t page_size, int32_t table_width, int64_t table_stride,
                               int32_t cache_type, int64_t k_stride, int64_t v_stride,
                               uint32_t *errors, ssd_stream_t stream)
{
    ssd::KvView c;
    const ssd_status_t st = ssd::kv_check(&c, k_cache, v_cache, k_scale, v_scale, query_start_loc,
                                          kv_lens, block_table, total_len, batch, nheads_kv,
                                          head_dim, num_pages, page_size, table_width,
                                          table_stride, cache_type, errors);
    if (st != SSD_OK)
        return st;
    return ssd::copy<false>(c, k, v, k_stride, v_stride, stream);
}

}  // extern "C"
