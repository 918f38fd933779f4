// Short causal convolution of every channel over a ragged batch:
//
//     y[t,c] = act(bias[c] + sum_{j < W} w[c,j] u[t - (W-1) + j, c])
//
// with u = x in the sequence and its slot's inputs before it.  One pass, bound by
// memory: x is read and y written once, two bytes each, against 2 W flops and the
// two special functions of silu.
//
// Work is done by warps on 128 channels, four a lane.  A warp either walks the rows
// of a tile of 32 with the last W - 1 rows in registers, whichever sequences they
// are of, and leaves out the first W - 1 tokens of each sequence; or it takes one
// sequence, does those first tokens and moves its slot on.  So a slot is read and
// written by one warp alone, and a batch of single tokens is all of the second kind.
//
// Width 4 with silu: four prompts of 22,500 tokens in all, 10,240 channels, 137.5 us, 98 % of the
// measured copy rate (with four rows ahead and seven CTAs of four warps 142 us, eight channels
// a lane 160); 100 single tokens and 156 of up to 127, 4,352 channels, 33.1 us.
#include "attn_ptx.cuh"
#include "layer_common.cuh"

namespace ssd {
namespace {

constexpr int kConvWarps = 2;         // warps of a CTA
constexpr int kConvResident = 11;     // CTAs of an SM
constexpr int kConvRows = 32;         // rows of a tile (the bits of a mask)
constexpr int kConvAhead = 8;         // rows that a warp loads at once, one such step ahead

struct ConvParams {
    SlotBatch s;
    __nv_bfloat16 *y;
    const __nv_bfloat16 *x;
    const float *weight, *bias;
    __nv_bfloat16 *pool;
    int64_t y_stride, x_stride;
    int32_t channels, blocks, tiles;  // blocks of 128 channels, tiles of rows
};

// Which rows of the tile at t0 take their inputs from x alone: bit i is set for row
// t0 + i unless it is one of the first kWidth - 1 of its sequence or behind the last
// sequence.  By a whole warp, a sequence a lane.
template <int kWidth>
__device__ __forceinline__ uint32_t rows_within(const SlotBatch &s, int64_t t0)
{
    const int lane = threadIdx.x & 31;
    uint32_t out = 0;
    for (int b = warp_last_start(s.qsl, s.batch, t0);; b += 32) {
        const int mine = b + lane;
        const int64_t at = mine <= s.batch ? s.qsl[mine] - t0 : kConvRows;
        if (at < kConvRows) {
            const uint32_t rows = mine == s.batch ? 0xffffffffu : (1u << (kWidth - 1)) - 1;
            if (at >= 0)
                out |= rows << at;
            else if (mine == s.batch)
                out = rows;
            else if (at > -32)
                out |= rows >> -at;
        }
        // (offsets that fall are an error: nothing is promised of their rows)
        if (__any_sync(0xffffffffu, mine >= s.batch || at >= kConvRows))
            break;
    }
    return ~__reduce_or_sync(0xffffffffu, out);
}

// Four values of a row, or a weight of four channels: two fp32 in a register pair.
struct Four {
    uint64_t v[2];
};

__device__ __forceinline__ Four widen_pairs(const uint2 &r)
{
    const uint32_t w[2] = {r.x, r.y};
    Four x;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        x.v[i] = ptx::pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    return x;
}

template <int kWidth>
struct ConvWeights {
    Four w[kWidth], bias;
    uint64_t log2e, one;

    __device__ __forceinline__ void load(const ConvParams &p, int c)
    {
        float flat[4 * kWidth];
#pragma unroll
        for (int i = 0; i < kWidth; ++i)
            *reinterpret_cast<float4 *>(flat + 4 * i) =
                __ldg(reinterpret_cast<const float4 *>(p.weight + static_cast<int64_t>(c) * kWidth) + i);
#pragma unroll
        for (int j = 0; j < kWidth; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                w[j].v[i] = ptx::pack2(flat[2 * i * kWidth + j], flat[(2 * i + 1) * kWidth + j]);
        const float4 v = p.bias ? __ldg(reinterpret_cast<const float4 *>(p.bias + c)) : make_float4(0, 0, 0, 0);
        bias.v[0] = ptx::pack2(v.x, v.y);
        bias.v[1] = ptx::pack2(v.z, v.w);
        log2e = ptx::pack2(-1.4426950408889634f, -1.4426950408889634f);
        one = ptx::pack2(1.f, 1.f);
    }

    // y of the row whose inputs are in[0] (the oldest) to in[kWidth - 1]
    template <bool kSilu>
    __device__ __forceinline__ uint2 row(const Four (&in)[kWidth]) const
    {
        uint32_t out[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint64_t v = bias.v[i];
#pragma unroll
            for (int j = 0; j < kWidth; ++j)
                v = ptx::fma2(w[j].v[i], in[j].v[i], v);
            if constexpr (kSilu) {
                float t0, t1, q0, q1;
                ptx::unpack2(ptx::mul2(v, log2e), t0, t1);
                ptx::unpack2(ptx::add2(ptx::pack2(ptx::ex2(t0), ptx::ex2(t1)), one), q0, q1);
                v = ptx::mul2(v, ptx::pack2(rcp_f32(q0), rcp_f32(q1)));
            }
            float a, b;
            ptx::unpack2(v, a, b);
            out[i] = pack_bf16(a, b);
        }
        return make_uint2(out[0], out[1]);
    }
};

template <int kWidth>
__device__ __forceinline__ void shift_in(Four (&in)[kWidth], const uint2 &raw)
{
#pragma unroll
    for (int j = 0; j + 1 < kWidth; ++j)
        in[j] = in[j + 1];
    in[kWidth - 1] = widen_pairs(raw);
}

template <int kWidth, bool kSilu>
__global__ void __launch_bounds__(kConvWarps * 32, kConvResident) conv_kernel(const __grid_constant__ ConvParams p)
{
    const int lane = threadIdx.x & 31;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kConvWarps + (threadIdx.x >> 5);
    const int job = static_cast<int>(item / p.blocks);
    const int c = (static_cast<int>(item % p.blocks) * 32 + lane) * 4;
    const bool mine = c < p.channels;
    pdl_wait();
    if (job >= p.tiles + p.s.batch)
        return;
    ConvWeights<kWidth> w;
    Four in[kWidth];
    auto x_row = [&](int64_t t) { return *reinterpret_cast<const uint2 *>(p.x + t * p.x_stride + c); };
    auto put = [&](int64_t t, const uint2 &v) { *reinterpret_cast<uint2 *>(p.y + t * p.y_stride + c) = v; };
    const uint2 none = make_uint2(0, 0);

    if (job < p.tiles) {
        const int64_t t0 = static_cast<int64_t>(job) * kConvRows, left = p.s.total_len - t0;
        // the rows do not depend on whose they are: the first ones are on their way
        uint2 before[kWidth - 1], raw[kConvAhead], next[kConvAhead];
#pragma unroll
        for (int j = 0; j + 1 < kWidth; ++j) {
            const int64_t t = t0 - (kWidth - 1) + j;
            before[j] = mine && t >= 0 ? x_row(t) : none;
        }
        auto fetch = [&](uint2 (&to)[kConvAhead], int i0) {
#pragma unroll
            for (int i = 0; i < kConvAhead; ++i)
                to[i] = mine && i0 + i < left && i0 < kConvRows ? x_row(t0 + i0 + i) : none;
        };
        fetch(raw, 0);
        uint32_t rows = rows_within<kWidth>(p.s, t0);
        if (left < 32)
            rows &= (1u << left) - 1;
        if (rows == 0 || !mine)
            return;
        w.load(p, c);
#pragma unroll
        for (int j = 0; j + 1 < kWidth; ++j)
            shift_in(in, before[j]);
        if (rows == 0xffffffffu) {
            // all of the tile's rows, as a rule: no tests, addresses go by steps
            const __nv_bfloat16 *xp = p.x + (t0 + kConvAhead) * p.x_stride + c;
            __nv_bfloat16 *yp = p.y + t0 * p.y_stride + c;
#pragma unroll 2
            for (int i0 = 0; i0 < kConvRows; i0 += kConvAhead) {
                if (i0 + kConvAhead < kConvRows) {
#pragma unroll
                    for (int i = 0; i < kConvAhead; ++i) {
                        next[i] = *reinterpret_cast<const uint2 *>(xp);
                        xp += p.x_stride;
                    }
                }
#pragma unroll
                for (int i = 0; i < kConvAhead; ++i) {
                    shift_in(in, raw[i]);
                    *reinterpret_cast<uint2 *>(yp) = w.template row<kSilu>(in);
                    yp += p.y_stride;
                    raw[i] = next[i];
                }
            }
            return;
        }
        for (int i0 = 0; i0 < kConvRows; i0 += kConvAhead) {
            fetch(next, i0 + kConvAhead);
#pragma unroll
            for (int i = 0; i < kConvAhead; ++i) {
                shift_in(in, raw[i]);
                if (rows >> (i0 + i) & 1)
                    put(t0 + i0 + i, w.template row<kSilu>(in));
                raw[i] = next[i];
            }
        }
        return;
    }

    const int b = job - p.tiles;
    int32_t begin, end;
    if (!seq_rows(p.s.qsl, p.s.total_len, p.s.errors, b, begin, end) || !mine)
        return;
    const int64_t slot = seq_slot(p.s, b);
    const bool has = slot >= 0 && p.s.has_init && p.s.has_init[b];
    __nv_bfloat16 *state = p.pool + slot * (kWidth - 1) * static_cast<int64_t>(p.channels) + c;
    const int len = end - begin;
    // the line of inputs: the slot's, then the sequence's
    uint2 old[kWidth - 1], first[kWidth - 1], last[kWidth - 1];
#pragma unroll
    for (int j = 0; j + 1 < kWidth; ++j) {
        old[j] = has ? *reinterpret_cast<const uint2 *>(state + static_cast<int64_t>(j) * p.channels) : none;
        first[j] = j < len ? x_row(begin + j) : none;
        last[j] = len + j >= kWidth - 1 ? x_row(begin + len + j - (kWidth - 1)) : none;
    }
    w.load(p, c);
#pragma unroll
    for (int j = 0; j + 1 < kWidth; ++j)
        shift_in(in, old[j]);
#pragma unroll
    for (int i = 0; i + 1 < kWidth; ++i) {
        shift_in(in, first[i]);
        if (i < len)
            put(begin + i, w.template row<kSilu>(in));
    }
    if (slot >= 0) {
#pragma unroll
        for (int j = 0; j + 1 < kWidth; ++j) {
            uint2 v = last[j];
#pragma unroll
            for (int k = 0; k + 1 < kWidth; ++k)
                if (len + j == k)
                    v = old[k];
            *reinterpret_cast<uint2 *>(state + static_cast<int64_t>(j) * p.channels) = v;
        }
    }
}

template <int kWidth>
cudaError_t launch_conv(const ConvParams &p, bool silu, dim3 grid, cudaStream_t stream)
{
    return launch_pdl(silu ? conv_kernel<kWidth, true> : conv_kernel<kWidth, false>, grid, kConvWarps * 32, stream, p);
}

}  // namespace
}  // namespace ssd

extern "C" ssd_status_t ssd_causal_conv_varlen_fwd(
    void *y, const void *x, const float *weight, const float *bias, void *conv_pool,
    const int32_t *query_start_loc, const uint8_t *has_initial_state,
    const uint32_t *cache_indices, int64_t total_len, int32_t batch, int32_t channels,
    int32_t width, int64_t max_slots, int64_t y_stride, int64_t x_stride, int32_t silu,
    uint32_t *errors, ssd_stream_t stream)
{
    using namespace ssd;
    ConvParams p = {};
    const ssd_status_t st = slots_check(&p.s, query_start_loc, has_initial_state, cache_indices,
                                        total_len, batch, max_slots, errors);
    if (st != SSD_OK)
        return st;
    if (channels <= 0 || width <= 0)
        return SSD_ERR_INVALID_ARG;
    if (channels % 8 != 0 || channels > (1 << 20) || width < 2 || width > 4)
        return SSD_ERR_UNSUPPORTED;
    if (!kv_pitch(&y_stride, channels) || !kv_pitch(&x_stride, channels))
        return SSD_ERR_INVALID_ARG;
    if (batch == 0)
        return SSD_OK;
    if ((total_len > 0 && (!y || !x)) || !weight || (max_slots > 0 && !conv_pool) || !kv_aligned16(y) ||
        !kv_aligned16(x) || !kv_aligned16(weight) || !kv_aligned16(bias) || !kv_aligned16(conv_pool))
        return SSD_ERR_INVALID_ARG;
    p.y = static_cast<__nv_bfloat16 *>(y);
    p.x = static_cast<const __nv_bfloat16 *>(x);
    p.weight = weight;
    p.bias = bias;
    p.pool = static_cast<__nv_bfloat16 *>(conv_pool);
    p.y_stride = y_stride;
    p.x_stride = x_stride;
    p.channels = channels;
    p.blocks = (channels + 127) / 128;
    p.tiles = static_cast<int32_t>((total_len + kConvRows - 1) / kConvRows);
    const int64_t items = (static_cast<int64_t>(p.tiles) + batch) * p.blocks;
    const int64_t ctas = (items + kConvWarps - 1) / kConvWarps;
    if (ctas > INT32_MAX)
        return SSD_ERR_UNSUPPORTED;
    const dim3 grid(static_cast<unsigned>(ctas));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = width == 4   ? launch_conv<4>(p, silu != 0, grid, s)
                          : width == 3 ? launch_conv<3>(p, silu != 0, grid, s)
                                       : launch_conv<2>(p, silu != 0, grid, s);
    return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}
