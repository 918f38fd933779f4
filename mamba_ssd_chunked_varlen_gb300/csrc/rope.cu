// Rotary positions of queries and keys, alone or with the write of the rotated keys
// and of the values into the paged cache:
//
//     (a, b) -> magnitude (a cos - b sin, b cos + a sin)  at the angle p f
//
// The angle.  In turns, f is a 64-bit binary fraction F / 2^64 (ssd_rope_table), and
// p F modulo 2^64 is p f modulo a turn, off by 2^-65 p alone.  Its upper 32 bits, read as
// signed, are an angle of at most half a turn, which sincospi takes without any
// reduction: 2^-33 turns, a rounding to fp32 (2^-24 of at most half a turn) and the
// function's own error are all there is, at any position.
//
// A warp takes a token: each lane two angles, which go through shared memory to the
// lanes that need them and serve all heads.  A row is head_dim / 8 lanes of eight
// elements, as in kv_cache.cu; a half's partner comes from another lane by shuffles.
#include <cmath>

#include "layer_common.cuh"

namespace ssd {
namespace {

constexpr int kRopeWarps = 8;         // tokens of a CTA
constexpr int kRopeAhead = 4;         // rows that a lane has in flight
constexpr int kRopeNone = -1;         // cache type of the call without a cache

struct RopeParams {
    KvView c;                         // without a cache: the batch, errors and the heads alone
    __nv_bfloat16 *q_out, *k_out;
    const __nv_bfloat16 *q, *k, *v;
    const uint64_t *turns;
    int64_t q_out_stride, q_stride, k_out_stride, k_stride, v_stride;
    int32_t heads, rows, part_rows;   // query heads; rows of a token, of them in one part
    int32_t part, half;               // rotated elements of a head, and half of them
    float magnitude;
};

// Position of row t of sequence b; negative: none.
template <int kType>
__device__ __forceinline__ int64_t position_of(const RopeParams &p, int b, int64_t t)
{
    int32_t begin, end;
    if (p.c.batch == 0 || !seq_rows(p.c.qsl, p.c.total_len, p.c.errors, b, begin, end) || t < begin || t >= end)
        return -1;
    if constexpr (kType == kRopeNone) {
        const int32_t n = p.c.kv_lens[b];
        if (n < 0)
            kv_error(p.c, SSD_DEVERR_BAD_KV_LEN);
        return n - static_cast<int64_t>(end) + t;
    } else {
        return kv_len_of(p.c, b) - static_cast<int64_t>(end) + t;
    }
}

// Cosines and sines of the pairs of a lane's eight elements.
template <bool kNeighbours>
struct LaneTurns {
    static constexpr int kPairs = kNeighbours ? 4 : 8;
    float cos[kPairs], sin[kPairs];

    // halves: the lower element's sine with its sign, a' = a cos - b sin
    __device__ __forceinline__ void load(const float2 *turn, int col, int half)
    {
        const int at = kNeighbours ? col / 2 : col % half;
        const float sign = !kNeighbours && col < half ? -1.f : 1.f;
#pragma unroll
        for (int i = 0; i < kPairs; i += 2) {
            const float4 two = *reinterpret_cast<const float4 *>(turn + at + i);
            cos[i] = two.x;
            sin[i] = sign * two.y;
            cos[i + 1] = two.z;
            sin[i + 1] = sign * two.w;
        }
    }

    __device__ __forceinline__ void rotate(float (&x)[8], const float (&partner)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            if constexpr (kNeighbours) {
                const float a = x[i], b = x[i + 1];
                x[i] = a * cos[i / 2] - b * sin[i / 2];
                x[i + 1] = b * cos[i / 2] + a * sin[i / 2];
            } else {
                x[i] = x[i] * cos[i] + partner[i] * sin[i];
                x[i + 1] = x[i + 1] * cos[i + 1] + partner[i + 1] * sin[i + 1];
            }
        }
    }
};

template <int kType, int kDim, bool kNeighbours>
__global__ void __launch_bounds__(kRopeWarps * 32) rope_kernel(const __grid_constant__ RopeParams p)
{
    constexpr int kLanes = kDim / 8;           // lanes of a row
    constexpr int kAtOnce = 32 / kLanes;       // rows of the warp's one load
    constexpr int kStep = kAtOnce * kRopeAhead;
    __shared__ alignas(16) float2 s_turn[kRopeWarps][kDim / 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    if (blockIdx.x == 0 && blockIdx.y == 0) {   // one CTA looks the offsets over
        int32_t begin, end;
        for (int b = threadIdx.x; b < p.c.batch; b += kRopeWarps * 32)
            seq_rows(p.c.qsl, p.c.total_len, p.c.errors, b, begin, end);
    }
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kRopeWarps + warp;
    if (t >= p.c.total_len)
        return;
    const int sub = lane / kLanes, col = (lane % kLanes) * 8;
    const int first = blockIdx.y * p.part_rows, last = min(first + p.part_rows, p.rows);
    const int q_rows = p.heads, k_rows = q_rows + p.c.heads;   // rows of q, then of k, then of v
    auto load = [&](int r) {
        if (r >= last)
            return make_uint4(0, 0, 0, 0);
        const __nv_bfloat16 *src = r < q_rows   ? p.q + t * p.q_stride + static_cast<int64_t>(r) * kDim
                                   : r < k_rows ? p.k + t * p.k_stride + static_cast<int64_t>(r - q_rows) * kDim
                                                : p.v + t * p.v_stride + static_cast<int64_t>(r - k_rows) * kDim;
        return *reinterpret_cast<const uint4 *>(src + col);
    };
    // the rows do not depend on their position: the first ones are on their way
    uint4 raw[kRopeAhead];
#pragma unroll
    for (int i = 0; i < kRopeAhead; ++i)
        raw[i] = load(first + i * kAtOnce + sub);

    const int b = warp_last_start(p.c.qsl, p.c.batch, t);
    const int64_t pos = position_of<kType>(p, b, t);
    if (pos < 0)
        return;
    for (int i = lane; i < p.half; i += 32) {
        const uint64_t turn = static_cast<uint64_t>(pos) * p.turns[i];
        // (adding half of the last bit kept rounds, and may carry into a whole turn)
        const int32_t angle = static_cast<int32_t>(static_cast<uint32_t>((turn + 0x80000000u) >> 32));
        float sin, cos;
        sincospif(static_cast<float>(angle) * 0x1p-31f, &sin, &cos);
        s_turn[warp][i] = make_float2(cos * p.magnitude, sin * p.magnitude);
    }
    int64_t page = -1;
    if constexpr (kType != kRopeNone)
        if (last > q_rows)
            page = kv_page_of(p.c, b, static_cast<int32_t>(pos));
    __syncwarp();
    LaneTurns<kNeighbours> turns;
    const bool turned = col < p.part;
    turns.load(s_turn[warp], turned ? col : 0, p.half);
    const int partner = kNeighbours || !turned ? lane : col < p.half ? lane + p.half / 8 : lane - p.half / 8;

    for (int r0 = first; r0 < last; r0 += kStep) {
        uint4 next[kRopeAhead];
#pragma unroll
        for (int i = 0; i < kRopeAhead; ++i)
            next[i] = load(r0 + kStep + i * kAtOnce + sub);
#pragma unroll
        for (int i = 0; i < kRopeAhead; ++i) {
            const int r = r0 + i * kAtOnce + sub;
            float x[8], other[8];
            widen8(raw[i], x);
            if constexpr (!kNeighbours) {
                uint4 o;
                o.x = __shfl_sync(0xffffffffu, raw[i].x, partner);
                o.y = __shfl_sync(0xffffffffu, raw[i].y, partner);
                o.z = __shfl_sync(0xffffffffu, raw[i].z, partner);
                o.w = __shfl_sync(0xffffffffu, raw[i].w, partner);
                widen8(o, other);
            }
            if (turned && r < k_rows)
                turns.rotate(x, other);
            if (r < q_rows) {
                if (r < last)
                    *reinterpret_cast<uint4 *>(p.q_out + t * p.q_out_stride + static_cast<int64_t>(r) * kDim +
                                               col) = round8(x);
            } else if constexpr (kType == kRopeNone) {
                if (r < last)
                    *reinterpret_cast<uint4 *>(p.k_out + t * p.k_out_stride +
                                               static_cast<int64_t>(r - q_rows) * kDim + col) = round8(x);
            }
            if constexpr (kType != kRopeNone) {
                const bool is_v = r >= k_rows, put = r >= q_rows && r < last && page >= 0;
                const int64_t row = kv_row(p.c, page, r - (is_v ? k_rows : q_rows), static_cast<int32_t>(pos));
                if constexpr (kType == SSD_KV_BF16) {
                    if (put)
                        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(is_v ? p.c.v : p.c.k) +
                                                   row * kDim + col) = is_v ? raw[i] : round8(x);
                } else {
                    constexpr float kTop = kType == SSD_KV_INT8 ? kInt8Max : kE4m3Max;
                    // magnitudes order as integers, infinities and NaN come last
                    uint32_t top = 0;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        top = max(top, __float_as_uint(x[k]) & 0x7fffffffu);
#pragma unroll
                    for (int o = 1; o < kLanes; o <<= 1)
                        top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                    if (put) {
                        const bool bad = top >= 0x7f800000u;
                        const float a = fmaxf(__uint_as_float(top), kKvTiny);
                        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(is_v ? p.c.v : p.c.k) + row * kDim +
                                                   col) =
                            bad ? make_uint2(0, 0) : encode8<kType>(x, __fdiv_rn(kTop, a));
                        if (col == 0)
                            (is_v ? p.c.v_scale : p.c.k_scale)[row] =
                                bad ? __int_as_float(0x7fffffff) : __fdiv_rn(a, kTop);
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kRopeAhead; ++i)
            raw[i] = next[i];
    }
}

template <int kType>
cudaError_t launch(RopeParams &p, int64_t total_len, bool neighbours, cudaStream_t stream)
{
    // a warp takes all of a token's rows once that gives every SM 16 warps; few tokens
    // are spread over warps, a load's rows each
    const int step = 256 / p.c.dim * kRopeAhead;
    const bool many = total_len >= 16 * 152;
    p.part_rows = many ? p.rows : step;
    const dim3 grid(static_cast<unsigned>((total_len + kRopeWarps - 1) / kRopeWarps),
                    static_cast<unsigned>((p.rows + p.part_rows - 1) / p.part_rows));
    const int threads = kRopeWarps * 32;
    if (p.c.dim == 128)
        return neighbours ? launch_pdl(rope_kernel<kType, 128, true>, grid, threads, stream, p)
                          : launch_pdl(rope_kernel<kType, 128, false>, grid, threads, stream, p);
    return neighbours ? launch_pdl(rope_kernel<kType, 64, true>, grid, threads, stream, p)
                      : launch_pdl(rope_kernel<kType, 64, false>, grid, threads, stream, p);
}

// What both calls check of the rotation; SSD_OK and p's fields set.
ssd_status_t rotation(RopeParams *p, const uint64_t *turns, int32_t head_dim, int32_t rotary_dim, float magnitude)
{
    if (rotary_dim <= 0 || rotary_dim > head_dim || !std::isfinite(magnitude))
        return SSD_ERR_INVALID_ARG;
    if (rotary_dim % 16 != 0 || (head_dim != 64 && head_dim != 128))
        return SSD_ERR_UNSUPPORTED;
    if (!turns || (reinterpret_cast<uintptr_t>(turns) & 7u) != 0)
        return SSD_ERR_INVALID_ARG;
    p->turns = turns;
    p->part = rotary_dim;
    p->half = rotary_dim / 2;
    p->magnitude = magnitude;
    return SSD_OK;
}

}  // namespace
}  // namespace ssd

extern "C" {

ssd_status_t ssd_rope_table(uint64_t *turns, const double *frequencies, int32_t n)
{
    // 1 / (2 pi) in two doubles: the product is right to some 2^-100
    constexpr double kHigh = 0x1.45f306dc9c883p-3, kLow = -0x1.6b01ec5417056p-57;
    if (n < 0 || (n > 0 && (!turns || !frequencies)))
        return SSD_ERR_INVALID_ARG;
    for (int32_t i = 0; i < n; ++i) {
        const double f = frequencies[i];
        if (!(f >= 0.0 && f < 6.283185307179586))
            return SSD_ERR_INVALID_ARG;
        const double high = f * kHigh, low = std::fma(f, kHigh, -high) + f * kLow;
        // high 2^64 is a whole number, or small enough that its fraction goes with low's
        const double scaled = std::ldexp(high, 64), whole = std::floor(scaled);
        const double rest = (scaled - whole) + std::ldexp(low, 64);
        turns[i] = (whole >= 0x1p64 ? 0u : static_cast<uint64_t>(whole)) +
                   static_cast<uint64_t>(static_cast<int64_t>(std::nearbyint(rest)));
    }
    return SSD_OK;
}

ssd_status_t ssd_rope_varlen_fwd(void *q_out, const void *q, void *k_out, const void *k,
                                 const uint64_t *turns, const int32_t *query_start_loc,
                                 const int32_t *kv_lens, int64_t total_len, int32_t batch,
                                 int32_t nheads, int32_t nheads_kv, int32_t head_dim,
                                 int32_t rotary_dim, int32_t interleaved, float magnitude,
                                 int64_t q_out_stride, int64_t q_stride, int64_t k_out_stride,
                                 int64_t k_stride, uint32_t *errors, ssd_stream_t stream)
{
    using namespace ssd;
    RopeParams p = {};
    if (total_len < 0 || batch < 0 || nheads < 0 || nheads_kv < 0 || nheads + int64_t{nheads_kv} == 0 || head_dim <= 0)
        return SSD_ERR_INVALID_ARG;
    if (total_len > INT32_MAX / 2 || batch > INT32_MAX / 2 || nheads > kKvMaxHeads || nheads_kv > kKvMaxHeads)
        return SSD_ERR_UNSUPPORTED;
    const ssd_status_t st = rotation(&p, turns, head_dim, rotary_dim, magnitude);
    if (st != SSD_OK)
        return st;
    const int64_t q_row = static_cast<int64_t>(nheads) * head_dim, k_row = static_cast<int64_t>(nheads_kv) * head_dim;
    if (!kv_pitch(&q_out_stride, q_row) || !kv_pitch(&q_stride, q_row) || !kv_pitch(&k_out_stride, k_row) ||
        !kv_pitch(&k_stride, k_row))
        return SSD_ERR_INVALID_ARG;
    if (total_len == 0 || batch == 0)
        return SSD_OK;
    if ((nheads > 0 && (!q || !q_out)) || (nheads_kv > 0 && (!k || !k_out)) || !query_start_loc || !kv_lens ||
        !kv_aligned16(q) || !kv_aligned16(q_out) || !kv_aligned16(k) || !kv_aligned16(k_out))
        return SSD_ERR_INVALID_ARG;
    p.c.qsl = query_start_loc;
    p.c.kv_lens = kv_lens;
    p.c.total_len = total_len;
    p.c.errors = errors;
    p.c.batch = batch;
    p.c.heads = nheads_kv;
    p.c.dim = head_dim;
    p.q_out = static_cast<__nv_bfloat16 *>(q_out);
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k_out = static_cast<__nv_bfloat16 *>(k_out);
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.q_out_stride = q_out_stride;
    p.q_stride = q_stride;
    p.k_out_stride = k_out_stride;
    p.k_stride = k_stride;
    p.heads = nheads;
    p.rows = nheads + nheads_kv;
    const cudaError_t e =
        launch<kRopeNone>(p, total_len, interleaved != 0, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status_t ssd_rope_kv_cache_write(
    void *q_out, const void *q, const void *k, const void *v, const uint64_t *turns, void *k_cache,
    void *v_cache, float *k_scale, float *v_scale, const int32_t *query_start_loc,
    const int32_t *kv_lens, const int32_t *block_table, int64_t total_len, int32_t batch,
    int32_t nheads, int32_t nheads_kv, int32_t head_dim, int32_t rotary_dim, int32_t interleaved,
    float magnitude, int64_t num_pages, int32_t page_size, int32_t table_width,
    int64_t table_stride, int32_t cache_type, int64_t q_out_stride, int64_t q_stride,
    int64_t k_stride, int64_t v_stride, uint32_t *errors, ssd_stream_t stream)
{
    using namespace ssd;
    RopeParams p = {};
    ssd_status_t st = kv_check(&p.c, k_cache, v_cache, k_scale, v_scale, query_start_loc, kv_lens,
                               block_table, total_len, batch, nheads_kv, head_dim, num_pages, page_size,
                               table_width, table_stride, cache_type, errors);
    if (st != SSD_OK)
        return st;
    if (nheads <= 0)
        return SSD_ERR_INVALID_ARG;
    if (nheads > kKvMaxHeads)
        return SSD_ERR_UNSUPPORTED;
    st = rotation(&p, turns, head_dim, rotary_dim, magnitude);
    if (st != SSD_OK)
        return st;
    const int64_t q_row = static_cast<int64_t>(nheads) * head_dim, k_row = static_cast<int64_t>(nheads_kv) * head_dim;
    if (!kv_pitch(&q_out_stride, q_row) || !kv_pitch(&q_stride, q_row) || !kv_pitch(&k_stride, k_row) ||
        !kv_pitch(&v_stride, k_row))
        return SSD_ERR_INVALID_ARG;
    if (total_len == 0 || batch == 0)
        return SSD_OK;
    if (!q || !q_out || !k || !v || !kv_aligned16(q) || !kv_aligned16(q_out) || !kv_aligned16(k) || !kv_aligned16(v))
        return SSD_ERR_INVALID_ARG;
    p.q_out = static_cast<__nv_bfloat16 *>(q_out);
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.v = static_cast<const __nv_bfloat16 *>(v);
    p.q_out_stride = q_out_stride;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.heads = nheads;
    p.rows = nheads + 2 * nheads_kv;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool near = interleaved != 0;
    const cudaError_t e = cache_type == SSD_KV_BF16       ? launch<SSD_KV_BF16>(p, total_len, near, s)
                          : cache_type == SSD_KV_FP8_E4M3 ? launch<SSD_KV_FP8_E4M3>(p, total_len, near, s)
                                                          : launch<SSD_KV_INT8>(p, total_len, near, s);
    return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
