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
// elements, as in kv_cache.cu; a half's partner comes from another lane by shuffles.  Rows go
// in steps of one tensor, so that only those that become codes are looked through for
// their largest, and a step's loads are on their way while the one before is worked on.
//
// Memory bounds rows of bf16 (9,000 tokens of 16 and 16 heads of 64, 73 MB, 13.4 us, 80 % of the
// measured copy rate with the launch; 64 and 64 heads of 128 98 %), instructions those
// that become codes (7,787 tokens of 32 and 8 heads of 128 to int8 33 us, 176 MB: a q row's
// lane issues 34, a k or v row's 66, and a token's angle and place 540 a warp).
#include <algorithm>
#include <cmath>

#include "attn_ptx.cuh"
#include "layer_common.cuh"

namespace ssd {
namespace {

constexpr int kRopeWarps = 4;         // tokens of a CTA
constexpr int kRopeResident = 6;      // CTAs of an SM
constexpr int kRopeAhead = 4;         // rows that a lane has in flight
constexpr int kRopeNone = -1;         // cache type of the call without a cache

struct RopeParams {
    KvView c;                         // without a cache: the batch, errors and the heads alone
    __nv_bfloat16 *q_out, *k_out;
    const __nv_bfloat16 *q, *k, *v;
    const uint64_t *turns;
    int64_t q_out_stride, q_stride, k_out_stride, k_stride, v_stride;
    int32_t heads;                    // query heads
    int32_t steps, part_steps;        // steps of a token, of them in one part
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
    uint64_t cos[kPairs / 2], sin[kPairs / 2];

    // halves: the lower element's sine with its sign, a' = a cos - b sin
    __device__ __forceinline__ void load(const float2 *turn, int col, int half)
    {
        const int at = kNeighbours ? col / 2 : col % half;
        const float sign = !kNeighbours && col < half ? -1.f : 1.f;
#pragma unroll
        for (int i = 0; i < kPairs; i += 2) {
            const float4 two = *reinterpret_cast<const float4 *>(turn + at + i);
            cos[i / 2] = ptx::pack2(two.x, two.z);
            sin[i / 2] = ptx::pack2(sign * two.y, sign * two.w);
        }
    }

    // eight elements as pairs, and in the other layout those of the lane's partner
    __device__ __forceinline__ void rotate(uint64_t (&x)[4], const uint64_t (&partner)[4]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (kNeighbours) {
                float a, b, c0, c1, s0, s1;
                ptx::unpack2(x[i], a, b);
                ptx::unpack2(cos[i / 2], c0, c1);
                ptx::unpack2(sin[i / 2], s0, s1);
                const float c = i & 1 ? c1 : c0, s = i & 1 ? s1 : s0;
                x[i] = ptx::pack2(a * c - b * s, b * c + a * s);
            } else {
                x[i] = ptx::fma2(x[i], cos[i], ptx::mul2(partner[i], sin[i]));
            }
        }
    }
};

__device__ __forceinline__ void widen_pairs(const uint4 &r, uint64_t (&x)[4])
{
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] = ptx::pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}

enum RopeTensor { kQ, kK, kV };

template <int kType, int kDim, bool kNeighbours>
__global__ void __launch_bounds__(kRopeWarps * 32, kRopeResident) rope_kernel(const __grid_constant__ RopeParams p)
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
    const int first = blockIdx.y * p.part_steps, last = min(first + p.part_steps, p.steps);
    const int q_steps = (p.heads + kStep - 1) / kStep, k_steps = (p.c.heads + kStep - 1) / kStep;
    const __nv_bfloat16 *q = p.q + t * p.q_stride + col, *k = p.k + t * p.k_stride + col;
    const __nv_bfloat16 *v = p.v + t * p.v_stride + col;
    // a step's tensor, its first row there, and the rows of the tensor
    struct Step {
        RopeTensor tensor;
        int row, rows;
    };
    auto step_of = [&](int i) {
        return i < q_steps             ? Step{kQ, i * kStep, p.heads}
               : i < q_steps + k_steps ? Step{kK, (i - q_steps) * kStep, p.c.heads}
                                       : Step{kV, (i - q_steps - k_steps) * kStep, p.c.heads};
    };
    auto load = [&](uint4 (&raw)[kRopeAhead], int at) {
        const Step s = step_of(at);
        const __nv_bfloat16 *src = s.tensor == kQ ? q : s.tensor == kK ? k : v;
#pragma unroll
        for (int i = 0; i < kRopeAhead; ++i) {
            const int r = s.row + i * kAtOnce + sub;
            raw[i] = make_uint4(0, 0, 0, 0);
            if (at < last && r < s.rows)
                raw[i] = *reinterpret_cast<const uint4 *>(src + r * kDim);
        }
    };
    // the rows do not depend on their position: the first ones are on their way
    uint4 raw[kRopeAhead], next[kRopeAhead];
    load(raw, first);

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
    int64_t cache_row = -1;                    // of head 0, further heads are a page apart
    if constexpr (kType != kRopeNone)
        if (last > q_steps) {
            const int64_t page = kv_page_of(p.c, b, static_cast<int32_t>(pos));
            cache_row = page < 0 ? -1 : kv_row(p.c, page, 0, static_cast<int32_t>(pos));
        }
    __syncwarp();
    LaneTurns<kNeighbours> turns;
    const bool turned = col < p.part;
    turns.load(s_turn[warp], turned ? col : 0, p.half);
    const int partner = kNeighbours || !turned ? lane : col < p.half ? lane + p.half / 8 : lane - p.half / 8;

    auto rotated = [&](const uint4 &r, uint64_t (&x)[4]) {
        widen_pairs(r, x);
        uint64_t other[4] = {};
        if constexpr (!kNeighbours) {
            uint4 o;
            o.x = __shfl_sync(0xffffffffu, r.x, partner);
            o.y = __shfl_sync(0xffffffffu, r.y, partner);
            o.z = __shfl_sync(0xffffffffu, r.z, partner);
            o.w = __shfl_sync(0xffffffffu, r.w, partner);
            widen_pairs(o, other);
        }
        if (turned)
            turns.rotate(x, other);
    };
    auto round_pairs = [](const uint64_t (&x)[4]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            ptx::unpack2(x[i], a, b);
            w[i] = pack_bf16(a, b);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    };
    // rows of q, or of k without a cache: rotated and stored
    auto turn_rows = [&](__nv_bfloat16 *dst, int row, int rows) {
#pragma unroll
        for (int i = 0; i < kRopeAhead; ++i) {
            if (row + i * kAtOnce >= rows)     // (the same in all lanes)
                break;
            uint64_t x[4];
            rotated(raw[i], x);
            const int r = row + i * kAtOnce + sub;
            if (r < rows)
                *reinterpret_cast<uint4 *>(dst + r * kDim) = round_pairs(x);
        }
    };
    // rows of k, rotated, or of v into the cache
    auto keep_rows = [&](bool is_v, int row, int rows) {
#pragma unroll
        for (int i = 0; i < kRopeAhead; ++i) {
            if (row + i * kAtOnce >= rows)
                break;
            uint64_t x[4];
            if (is_v)
                widen_pairs(raw[i], x);
            else
                rotated(raw[i], x);
            const int r = row + i * kAtOnce + sub;
            const bool put = r < rows && cache_row >= 0;
            const int64_t to = cache_row + (static_cast<int64_t>(r) << p.c.page_shift);
            void *cache = is_v ? p.c.v : p.c.k;
            if constexpr (kType == SSD_KV_BF16) {
                if (put)
                    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(cache) + to * kDim + col) =
                        is_v ? raw[i] : round_pairs(x);
            } else if constexpr (kType != kRopeNone) {
                constexpr float kTop = kType == SSD_KV_INT8 ? kInt8Max : kE4m3Max;
                float f[8];
                // magnitudes order as integers, infinities and NaN come last
                uint32_t top = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    ptx::unpack2(x[j], f[2 * j], f[2 * j + 1]);
                    top = max(top, max(__float_as_uint(f[2 * j]) & 0x7fffffffu,
                                       __float_as_uint(f[2 * j + 1]) & 0x7fffffffu));
                }
#pragma unroll
                for (int o = 1; o < kLanes; o <<= 1)
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                const bool bad = top >= 0x7f800000u;
                const float a = fmaxf(__uint_as_float(top), kKvTiny);
                if (put) {
                    *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(cache) + to * kDim + col) =
                        bad ? make_uint2(0, 0) : encode8<kType>(f, __fdiv_rn(kTop, a));
                    if (col == 0)
                        (is_v ? p.c.v_scale : p.c.k_scale)[to] =
                            bad ? __int_as_float(0x7fffffff) : __fdiv_rn(a, kTop);
                }
            }
        }
    };
    for (int at = first; at < last; ++at) {
        load(next, at + 1);
        const Step s = step_of(at);
        if (s.tensor == kQ)
            turn_rows(p.q_out + t * p.q_out_stride + col, s.row, s.rows);
        else if constexpr (kType == kRopeNone)
            turn_rows(p.k_out + t * p.k_out_stride + col, s.row, s.rows);
        else
            keep_rows(s.tensor == kV, s.row, s.rows);
#pragma unroll
        for (int i = 0; i < kRopeAhead; ++i)
            raw[i] = next[i];
    }
}

template <int kType>
cudaError_t launch(RopeParams &p, int64_t total_len, bool neighbours, cudaStream_t stream)
{
    // a warp takes about three of a token's steps once that gives every SM 16 warps: enough for
    // the next one's loads to be ahead, and for a last wave that is not long (7,787 tokens of 32 and
    // 8 heads of 128 to int8, six steps, with the reading back: 49 us whole, 45.6 in two parts, 47
    // in three); few tokens are spread over warps, a step each
    const int step = 256 / p.c.dim * kRopeAhead, kv = (p.c.heads + step - 1) / step;
    p.steps = (p.heads + step - 1) / step + (kType == kRopeNone ? kv : 2 * kv);
    const int parts = std::max(1, (p.steps + 1) / 3);
    int device = 0, sms = 0;
    if (cudaGetDevice(&device) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
        return cudaErrorInvalidDevice;
    p.part_steps = total_len >= int64_t{16} * sms ? (p.steps + parts - 1) / parts : 1;
    const dim3 grid(static_cast<unsigned>((total_len + kRopeWarps - 1) / kRopeWarps),
                    static_cast<unsigned>((p.steps + p.part_steps - 1) / p.part_steps));
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
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool near = interleaved != 0;
    const cudaError_t e = cache_type == SSD_KV_BF16       ? launch<SSD_KV_BF16>(p, total_len, near, s)
                          : cache_type == SSD_KV_FP8_E4M3 ? launch<SSD_KV_FP8_E4M3>(p, total_len, near, s)
                                                          : launch<SSD_KV_INT8>(p, total_len, near, s);
    return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
