// Paged key/value cache: rows quantised as they are written, and read back.
//
// Write, per row x of head_dim elements (one token, one head, K or V):
//     a = max(max|x|, 2^-60),  code = round(x * (M / a)),  scale = a / M
// Read: x' = bf16(code * scale).  One pass over the rows in each direction.
#include <type_traits>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "attn_common.cuh"
#include "rows.cuh"
#include "ssd_device.cuh"

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
        static_cast<int64_t>(table_width) * page_size > INT32_MAX / 2 || nheads_kv > kKvMaxHeads)
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

template <int kType>
__device__ __forceinline__ void decode8(const uint2 &r, float (&x)[8])
{
    const uint32_t w[2] = {r.x, r.y};
    if constexpr (kType == SSD_KV_INT8) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = static_cast<float>(static_cast<int8_t>(w[i >> 2] >> (8 * (i & 3))));
    } else {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2(
                static_cast<__nv_fp8x2_storage_t>(w[i >> 2] >> (8 * (i & 3))), __NV_E4M3));
            const float2 f = __half22float2(h);
            x[i] = f.x;
            x[i + 1] = f.y;
        }
    }
}

// Where the rows of tokens [t, t + kTokens) lie, by a whole warp: lane i < kTokens
// gets token t + i's row of head 0 in the cache (rows of further heads are a page
// apart), or -1 when it has none.
template <int kTokens>
__device__ __forceinline__ int64_t place_tokens(const KvView &c, int64_t t)
{
    int b = warp_sequence_of(c, t);
    if constexpr (kTokens == 1) {
        if (b < 0)
            return -1;
        const int64_t j = kv_len_of(c, b) - static_cast<int64_t>(c.qsl[b + 1]) + t;
        const int64_t page = j < 0 ? -1 : kv_page_of(c, b, static_cast<int32_t>(j));
        return page < 0 ? -1 : kv_row(c, page, 0, static_cast<int32_t>(j));
    }
    const int lane = threadIdx.x & 31;
    const int64_t mine = t + lane;
    if (lane >= kTokens || mine >= c.total_len)
        return -1;
    if (b < 0 && lane > 0)      // the first is nobody's; the others look from the start
        b = 0;
    // (as a rule the tokens are of one sequence)
    while (b >= 0 && b + 1 < c.batch && static_cast<int64_t>(c.qsl[b + 1]) <= mine)
        ++b;
    if (b < 0 || static_cast<int64_t>(c.qsl[b]) > mine || static_cast<int64_t>(c.qsl[b + 1]) <= mine)
        return -1;
    const int64_t j = kv_len_of(c, b) - static_cast<int64_t>(c.qsl[b + 1]) + mine;
    const int64_t page = j < 0 ? -1 : kv_page_of(c, b, static_cast<int32_t>(j));
    return page < 0 ? -1 : kv_row(c, page, 0, static_cast<int32_t>(j));
}

// One warp: of kTokens tokens, K and V rows [first, first + 4 * 256 / dim) of the
// token's 2 * heads.  A row is dim / 8 lanes of eight elements.  Finding a token's
// place takes five loads in a row.  A write loads its rows meanwhile; a read has
// to wait, so that with many tokens a warp places four at once and has all of their
// rows in flight together, while a few tokens are spread over warps.  Memory bounds
// a long int8 read (403 MB of codes and rows in 65.3 us, 91 % of the copy rate; one
// token a warp 14 us more), the instructions per element a quantising write.
template <int kType, int kDim, bool kWrite, int kTokens>
__global__ void __launch_bounds__(kWarps * 32)
    kv_copy_kernel(const __grid_constant__ KvView c, __nv_bfloat16 *k, __nv_bfloat16 *v, int64_t k_stride,
                   int64_t v_stride)
{
    constexpr int kLanes = kDim / 8;           // lanes of a row
    constexpr int kAtOnce = 32 / kLanes;       // rows of the warp's one load
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * kTokens;
    if (blockIdx.x == 0 && blockIdx.y == 0) {   // one CTA looks the offsets over
        bool bad = false;
        for (int b = threadIdx.x; b < c.batch; b += kWarps * 32)
            bad = bad || c.qsl[b + 1] < c.qsl[b] || (b == 0 && c.qsl[0] != 0) ||
                  (b == c.batch - 1 && c.qsl[c.batch] != c.total_len);
        if (bad)
            kv_error(c, SSD_DEVERR_BAD_QUERY_START_LOC);
    }
    if (t0 >= c.total_len)
        return;
    const int sub = lane / kLanes, col = (lane % kLanes) * 8;
    const int first = blockIdx.y * (kAtOnce * kRowsPerLane) + sub;
    const int rows = 2 * c.heads;
    using Raw = std::conditional_t<kWrite || kType == SSD_KV_BF16, uint4, uint2>;
    Raw raw[kTokens][kRowsPerLane];
    float scale[kTokens][kRowsPerLane];
    auto each = [&](auto f) {     // f(token, row of the lane, is it V's, head)
#pragma unroll
        for (int n = 0; n < kTokens; ++n)
#pragma unroll
            for (int i = 0; i < kRowsPerLane; ++i) {
                const int r = first + i * kAtOnce;
                if (r < rows && t0 + n < c.total_len)
                    f(n, i, r >= c.heads, r >= c.heads ? r - c.heads : r);
            }
    };
    auto token_row = [&](int n, bool is_v, int head) {
        return (is_v ? v + (t0 + n) * v_stride : k + (t0 + n) * k_stride) + head * kDim + col;
    };
    if constexpr (kWrite)
        // the rows do not depend on where they go: their loads start first
        each([&](int n, int i, bool is_v, int head) {
            raw[n][i] = *reinterpret_cast<const uint4 *>(token_row(n, is_v, head));
        });
    const int64_t mine = place_tokens<kTokens>(c, t0);
    int64_t base[kTokens];
#pragma unroll
    for (int n = 0; n < kTokens; ++n)
        base[n] = __shfl_sync(0xffffffffu, mine, n);
    auto cache_row = [&](int n, int head) { return base[n] + (static_cast<int64_t>(head) << c.page_shift); };

    if constexpr (kWrite && kType == SSD_KV_BF16) {
        each([&](int n, int i, bool is_v, int head) {
            if (base[n] >= 0)
                *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(is_v ? c.v : c.k) +
                                           cache_row(n, head) * kDim + col) = raw[n][i];
        });
    } else if constexpr (kWrite) {
        constexpr float kTop = kType == SSD_KV_INT8 ? kInt8Max : kE4m3Max;
        static_assert(kTokens == 1 && kRowsPerLane == 4);
        // The largest magnitude of each row: bf16 bits without the sign order as
        // integers, and infinities and NaN come last.  Lane l of a row's lanes keeps
        // row l % 4's, so that one division serves a lane's four rows.
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 in = first + i * kAtOnce < rows ? raw[0][i] : make_uint4(0, 0, 0, 0);
            uint32_t m = __vmaxu2(__vmaxu2(in.x & 0x7fff7fffu, in.y & 0x7fff7fffu),
                                  __vmaxu2(in.z & 0x7fff7fffu, in.w & 0x7fff7fffu));
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1)
                m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
            if ((lane & 3) == i)
                top = m;
        }
        top = max(top >> 16, top & 0xffffu);
        const bool bad = top >= 0x7f80u;
        const float a = fmaxf(__uint_as_float(top << 16), kKvTiny);
        const float inv = bad ? -1.f : __fdiv_rn(kTop, a);
        const int mine_row = first + (lane & 3) * kAtOnce;
        if (base[0] >= 0 && lane % kLanes < 4 && mine_row < rows) {
            const bool is_v = mine_row >= c.heads;
            (is_v ? c.v_scale : c.k_scale)[cache_row(0, is_v ? mine_row - c.heads : mine_row)] =
                bad ? __int_as_float(0x7fffffff) : __fdiv_rn(a, kTop);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = first + i * kAtOnce;
            const float by = __shfl_sync(0xffffffffu, inv, i, 4);
            if (r < rows && base[0] >= 0) {
                const bool is_v = r >= c.heads;
                float x[8];
                widen8(raw[0][i], x);
                const uint2 w = by < 0.f ? make_uint2(0, 0) : encode8<kType>(x, by);
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(is_v ? c.v : c.k) +
                                           cache_row(0, is_v ? r - c.heads : r) * kDim + col) = w;
            }
        }
    } else {
        each([&](int n, int i, bool is_v, int head) {
            raw[n][i] = Raw{};
            scale[n][i] = 0.f;
            if (base[n] >= 0) {
                const int64_t row = cache_row(n, head);
                raw[n][i] = *reinterpret_cast<const Raw *>(static_cast<const uint8_t *>(is_v ? c.v : c.k) +
                                                           (row * kDim + col) * (sizeof(Raw) / 8));
                if constexpr (kType != SSD_KV_BF16)
                    scale[n][i] = (is_v ? c.v_scale : c.k_scale)[row];
            }
        });
        each([&](int n, int i, bool is_v, int head) {
            uint4 out;
            if constexpr (kType == SSD_KV_BF16) {
                out = raw[n][i];
            } else {
                float x[8];
                decode8<kType>(raw[n][i], x);
                const float s = scale[n][i];
                out = make_uint4(pack_bf16(x[0] * s, x[1] * s), pack_bf16(x[2] * s, x[3] * s),
                                 pack_bf16(x[4] * s, x[5] * s), pack_bf16(x[6] * s, x[7] * s));
            }
            *reinterpret_cast<uint4 *>(token_row(n, is_v, head)) = out;
        });
    }
}

template <int kType, int kDim, bool kWrite>
cudaError_t launch(const KvView &c, void *k, void *v, int64_t ks, int64_t vs, cudaStream_t stream)
{
    constexpr int kRows = 32 / (kDim / 8) * kRowsPerLane;
    const unsigned parts = (2 * c.heads + kRows - 1) / kRows;
    // reads: four tokens a warp once that still gives every SM 16 warps
    constexpr int kMany = kWrite ? 1 : 4;
    const bool many = c.total_len * parts >= kMany * 16 * 152;
    const int64_t tokens = kWarps * (many ? kMany : 1);
    const dim3 grid(static_cast<unsigned>((c.total_len + tokens - 1) / tokens), parts);
    __nv_bfloat16 *kk = static_cast<__nv_bfloat16 *>(k), *vv = static_cast<__nv_bfloat16 *>(v);
    return launch_pdl(many ? kv_copy_kernel<kType, kDim, kWrite, kMany> : kv_copy_kernel<kType, kDim, kWrite, 1>,
                      grid, kWarps * 32, stream, c, kk, vv, ks, vs);
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
