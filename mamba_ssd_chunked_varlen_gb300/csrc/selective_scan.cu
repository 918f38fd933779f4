// Selective scan over a ragged batch: every channel d has a step of its own and N
// states with decays of their own,
//
//     dt = softplus(dt_raw + dt_bias),   h_n = exp(dt A_n) h_n + dt x B_n
//     y = sum_n C_n h_n + D x,           y silu(z) with a gate
//
// The decays differ in every (channel, state), so the chunked products of the SSD scan do
// not apply: one exponential and four multiply-adds per (token, channel, state).
// Measured on this GPU, exponentials go at 4 cycles a warp and scheduler and two fp32
// multiply-adds (fma.rn.f32x2) at 2, so that both pipes are about equally loaded and
// the kernel is written to issue as little else as it can.
//
// A channel is N / 8 lanes of eight states, kept as pairs of fp32.  A warp is 32 N / 8
// channels on its own; its CTA shares the tokens' B and C, widened to fp32 in shared
// memory.  Tokens go in groups of eight: each of a channel's lanes makes the steps of
// its share of them and hands them over by shuffles, and gets the sums of its share
// back from a reduction that halves the sums as it halves the lanes.
#include <algorithm>

#include "layer_common.cuh"

namespace ssd {
namespace {

constexpr int kScanWarps = 4;
constexpr int kScanThreads = kScanWarps * 32;
constexpr int kStates = 8;            // states of a lane
constexpr int kGroup = 8;             // tokens of a group
constexpr int kBlock = 32;            // tokens whose B and C are in shared memory at once

struct SelParams {
    SlotBatch s;
    __nv_bfloat16 *y;
    const __nv_bfloat16 *x, *dt, *B, *C, *z;
    const float *A, *D, *dt_bias;
    void *pool;
    int64_t y_stride, x_stride, dt_stride, b_stride, c_stride, z_stride;
    int32_t channels, tiles;          // tiles of a CTA's channels
    int32_t softplus;
};

// ---------------------------------------------------------------- arithmetic
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 values in one register pair.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 pack2(float a, float b)
{
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(F2 a, float &x, float &y)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a.v));
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// max(v, 0) + log(1 + e^-|v|).  With e = e^-|v| in (0, 1], log(1 + e) = e P(e), P of degree
// 9 fitted to log(1 + e) / e (relative error 5e-9, 1.6e-7 with fp32's roundings): small
// steps keep their relative precision.
__device__ __forceinline__ float step_of(float v)
{
    const float e = ex2(-1.4426950408889634f * fabsf(v));
    float p = -0.0032440251670777798f;
    p = fmaf(p, e, 0.01985146291553974f);
    p = fmaf(p, e, -0.05695953220129013f);
    p = fmaf(p, e, 0.10603655129671097f);
    p = fmaf(p, e, -0.15305592119693756f);
    p = fmaf(p, e, 0.1967593878507614f);
    p = fmaf(p, e, -0.24954134225845337f);
    p = fmaf(p, e, 0.3332996368408203f);
    p = fmaf(p, e, -0.4999990165233612f);
    p = fmaf(p, e, 1.f);
    return fmaf(p, e, fmaxf(v, 0.f));
}

// ---------------------------------------------------------------- pool
template <bool kBf16>
__device__ __forceinline__ void load_states(const void *pool, int64_t at, F2 (&h)[kStates / 2])
{
    float v[8];
    if constexpr (kBf16) {
        widen8(*reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(pool) + at), v);
    } else {
        *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(static_cast<const float *>(pool) + at);
        *reinterpret_cast<float4 *>(v + 4) = *reinterpret_cast<const float4 *>(static_cast<const float *>(pool) + at + 4);
    }
#pragma unroll
    for (int k = 0; k < kStates / 2; ++k)
        h[k] = pack2(v[2 * k], v[2 * k + 1]);
}

template <bool kBf16>
__device__ __forceinline__ void store_states(void *pool, int64_t at, const F2 (&h)[kStates / 2])
{
    float v[8];
#pragma unroll
    for (int k = 0; k < kStates / 2; ++k)
        unpack2(h[k], v[2 * k], v[2 * k + 1]);
    if constexpr (kBf16) {
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(pool) + at) = round8(v);
    } else {
        *reinterpret_cast<float4 *>(static_cast<float *>(pool) + at) = *reinterpret_cast<const float4 *>(v);
        *reinterpret_cast<float4 *>(static_cast<float *>(pool) + at + 4) = *reinterpret_cast<const float4 *>(v + 4);
    }
}

// ---------------------------------------------------------------- a sequence
template <int N>
struct SelShared {
    float B[2][kBlock][N], C[2][kBlock][N];
};

// What one lane holds of its channel.
template <int N>
struct SelLane {
    static constexpr int kLanes = N / kStates;       // lanes of a channel
    static constexpr int kChannels = 32 / kLanes;    // channels of a warp
    static constexpr int kMine = kGroup / kLanes;    // tokens of a group that a lane makes the steps of

    const SelParams &p;
    int part, in_warp, ch;                           // states' part, channel in the warp, channel
    bool valid;
    F2 a[kStates / 2], h[kStates / 2];               // A log2(e), the states
    float D, bias;

    // one token: B and C in shared memory from this lane's part on; returns sum C h of the part
    __device__ __forceinline__ float token(float dt, float u, const float *B, const float *C)
    {
        const F2 dt2 = pack2(dt, dt), u2 = pack2(u, u);
        F2 sum = pack2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kStates / 2; k += 2) {
            const float4 b = *reinterpret_cast<const float4 *>(B + 2 * k);
            const float4 c = *reinterpret_cast<const float4 *>(C + 2 * k);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float e0, e1;
                unpack2(mul2(dt2, a[k + i]), e0, e1);
                const F2 in = mul2(u2, i ? pack2(b.z, b.w) : pack2(b.x, b.y));
                h[k + i] = fma2(pack2(ex2(e0), ex2(e1)), h[k + i], in);
                sum = fma2(h[k + i], i ? pack2(c.z, c.w) : pack2(c.x, c.y), sum);
            }
        }
        float s0, s1;
        unpack2(sum, s0, s1);
        return s0 + s1;
    }

    __device__ __forceinline__ float step(const __nv_bfloat16 raw) const
    {
        const float v = __bfloat162float(raw) + bias;
        return p.softplus ? step_of(v) : v;
    }

    __device__ __forceinline__ void put(int64_t t, float sum, float x, const __nv_bfloat16 z)
    {
        float v = fmaf(D, x, sum);
        if (p.z)
            v *= silu_f32(__bfloat162float(z));
        if (valid)
            p.y[t * p.y_stride + ch] = __float2bfloat16_rn(v);
    }
};

// Sums over a channel's lanes of kLanes tokens at once: lane part gets token part's.
template <int kLanes, int kChannels>
__device__ __forceinline__ float reduce_tokens(float (&v)[kLanes], int part)
{
#pragma unroll
    for (int n = kLanes / 2; n >= 1; n /= 2) {
        const bool upper = part & n;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float send = upper ? v[i] : v[i + n], keep = upper ? v[i + n] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, n * kChannels);
        }
    }
    return v[0];
}

template <int N, bool kBf16>
__global__ void __launch_bounds__(kScanThreads) selective_scan_kernel(const __grid_constant__ SelParams p)
{
    using Lane = SelLane<N>;
    constexpr int kLanes = Lane::kLanes, kChannels = Lane::kChannels, kMine = Lane::kMine;
    __shared__ alignas(16) SelShared<N> s;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.x / p.tiles, tile = blockIdx.x % p.tiles;
    Lane me{p, lane / kChannels, lane % kChannels};
    me.ch = (tile * kScanWarps + warp) * kChannels + me.in_warp;
    me.valid = me.ch < p.channels;
    const int ch = me.valid ? me.ch : 0;      // (the other lanes follow a channel that is there)
    pdl_wait();
    int32_t begin, end;
    if (!seq_rows(p.s.qsl, p.s.total_len, p.s.errors, b, begin, end))
        return;
    const int64_t slot = seq_slot(p.s, b);
    const bool has = slot >= 0 && p.s.has_init && p.s.has_init[b];
    const int64_t at = (slot * p.channels + ch) * N + me.part * kStates;
#pragma unroll
    for (int k = 0; k < kStates / 2; ++k)
        me.h[k] = pack2(0.f, 0.f);
    if (has)
        load_states<kBf16>(p.pool, at, me.h);
    {
        const float *A = p.A + static_cast<int64_t>(ch) * N + me.part * kStates;
#pragma unroll
        for (int k = 0; k < kStates / 2; ++k) {
            const float2 v = __ldg(reinterpret_cast<const float2 *>(A) + k);
            me.a[k] = pack2(v.x * 1.4426950408889634f, v.y * 1.4426950408889634f);
        }
    }
    me.D = p.D ? p.D[ch] : 0.f;
    me.bias = p.dt_bias ? p.dt_bias[ch] : 0.f;

    // B and C of a block: one load of eight values at a time
    constexpr int kLoads = (2 * kBlock * N / 8 + kScanThreads - 1) / kScanThreads;
    uint4 bc[kLoads];
    auto fetch = [&](int t0) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int at = i * kScanThreads + threadIdx.x, row = at / (N / 8) % kBlock, col = at % (N / 8) * 8;
            const bool is_c = at >= kBlock * N / 8;
            bc[i] = make_uint4(0, 0, 0, 0);
            if (at < 2 * kBlock * N / 8 && t0 + row < end)
                bc[i] = *reinterpret_cast<const uint4 *>(
                    (is_c ? p.C + (t0 + row) * p.c_stride : p.B + (t0 + row) * p.b_stride) + col);
        }
    };
    auto stage = [&](int buffer) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int at = i * kScanThreads + threadIdx.x, row = at / (N / 8) % kBlock, col = at % (N / 8) * 8;
            if (at < 2 * kBlock * N / 8) {
                float v[8];
                widen8(bc[i], v);
                float *dst = (at >= kBlock * N / 8 ? s.C[buffer][row] : s.B[buffer][row]) + col;
                *reinterpret_cast<float4 *>(dst) = *reinterpret_cast<const float4 *>(v);
                *reinterpret_cast<float4 *>(dst + 4) = *reinterpret_cast<const float4 *>(v + 4);
            }
        }
    };
    const __nv_bfloat16 *px = p.x + ch, *pd = p.dt + ch, *pz = p.z ? p.z + ch : nullptr;
    // x, dt and z of the lane's tokens of a group
    __nv_bfloat16 x[kMine], d[kMine], z[kMine];
    auto load_group = [&](int t0) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int64_t t = t0 + i * kLanes + me.part;
            x[i] = d[i] = z[i] = __float2bfloat16_rn(0.f);
            if (t0 + kGroup <= end) {
                x[i] = px[t * p.x_stride];
                d[i] = pd[t * p.dt_stride];
                if (pz)
                    z[i] = pz[t * p.z_stride];
            }
        }
    };

    load_group(begin);
    fetch(begin);
    int buffer = 0;
    for (int t0 = begin; t0 < end; t0 += kBlock, buffer ^= 1) {
        stage(buffer);
        if (t0 + kBlock < end)
            fetch(t0 + kBlock);
        __syncthreads();   // (a warp that is ahead writes the other buffer)
        const float *B = s.B[buffer][0] + me.part * kStates, *C = s.C[buffer][0] + me.part * kStates;
        const int n = min(kBlock, end - t0);
        int g = 0;
        for (; g + kGroup <= n; g += kGroup) {
            float dt[kMine], u[kMine], xs[kMine];
            __nv_bfloat16 zs[kMine];
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                xs[i] = __bfloat162float(x[i]);
                zs[i] = z[i];
                dt[i] = me.step(d[i]);
                u[i] = dt[i] * xs[i];
            }
            load_group(t0 + g + kGroup);
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                float sums[kLanes];
#pragma unroll
                for (int j = 0; j < kLanes; ++j) {
                    const int from = j * kChannels + me.in_warp, row = (g + i * kLanes + j) * N;
                    const float dj = kLanes == 1 ? dt[i] : __shfl_sync(0xffffffffu, dt[i], from);
                    const float uj = kLanes == 1 ? u[i] : __shfl_sync(0xffffffffu, u[i], from);
                    sums[j] = me.token(dj, uj, B + row, C + row);
                }
                me.put(t0 + g + i * kLanes + me.part, reduce_tokens<kLanes, kChannels>(sums, me.part), xs[i], zs[i]);
            }
        }
        for (; g < n; ++g) {      // the last tokens, fewer than a group
            const int64_t t = t0 + g;
            const float xt = __bfloat162float(px[t * p.x_stride]), dt = me.step(pd[t * p.dt_stride]);
            float sum = me.token(dt, dt * xt, B + g * N, C + g * N);
#pragma unroll
            for (int o = kChannels; o < 32; o <<= 1)
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (me.part == 0)
                me.put(t, sum, xt, pz ? pz[t * p.z_stride] : __float2bfloat16_rn(0.f));
        }
    }
    if (slot >= 0 && me.valid)
        store_states<kBf16>(p.pool, at, me.h);
}

template <int N>
cudaError_t launch(SelParams &p, bool bf16, cudaStream_t stream)
{
    const int cols = kScanWarps * SelLane<N>::kChannels;
    p.tiles = (p.channels + cols - 1) / cols;
    const dim3 grid(static_cast<unsigned>(p.tiles * p.s.batch));
    return bf16 ? launch_pdl(selective_scan_kernel<N, true>, grid, kScanThreads, stream, p)
                : launch_pdl(selective_scan_kernel<N, false>, grid, kScanThreads, stream, p);
}

bool sel_sizes(int64_t total_len, int32_t batch, int32_t channels, int32_t dstate)
{
    return total_len >= 0 && total_len <= INT32_MAX / 2 && batch >= 0 && batch <= INT32_MAX / 2 && channels > 0 &&
           channels % 8 == 0 && channels <= (1 << 20) &&
           (dstate == 8 || dstate == 16 || dstate == 32 || dstate == 64) &&
           (static_cast<int64_t>(channels) + 7) / 8 * std::max<int64_t>(batch, 1) <= INT32_MAX;
}

}  // namespace
}  // namespace ssd

extern "C" {

size_t ssd_selective_scan_varlen_workspace_size(int64_t total_len, int32_t batch, int32_t channels,
                                                int32_t dstate)
{
    return ssd::sel_sizes(total_len, batch, channels, dstate) ? 256 : 0;
}

ssd_status_t ssd_selective_scan_varlen_fwd(
    void *y, const void *x, const void *dt, const float *A, const void *B, const void *C,
    const float *D, const void *z, const float *dt_bias, void *ssm_pool,
    const int32_t *query_start_loc, const uint8_t *has_initial_state,
    const uint32_t *cache_indices, int64_t total_len, int32_t batch, int32_t channels,
    int32_t dstate, int64_t max_slots, int32_t pool_type, int32_t dt_softplus,
    const ssd_selective_strides_t *strides, void *workspace, size_t workspace_bytes,
    uint32_t *errors, ssd_stream_t stream)
{
    using namespace ssd;
    SelParams p = {};
    const ssd_status_t st = slots_check(&p.s, query_start_loc, has_initial_state, cache_indices,
                                        total_len, batch, max_slots, errors);
    if (st != SSD_OK)
        return st;
    if (channels <= 0 || dstate <= 0 || (pool_type != SSD_POOL_FP32 && pool_type != SSD_POOL_BF16))
        return SSD_ERR_INVALID_ARG;
    if (!sel_sizes(total_len, batch, channels, dstate))
        return SSD_ERR_UNSUPPORTED;
    ssd_selective_strides_t t = {};
    if (strides)
        t = *strides;
    if (!kv_pitch(&t.y, channels) || !kv_pitch(&t.x, channels) || !kv_pitch(&t.dt, channels) ||
        !kv_pitch(&t.z, channels) || !kv_pitch(&t.B, dstate) || !kv_pitch(&t.C, dstate))
        return SSD_ERR_INVALID_ARG;
    if (batch == 0)
        return SSD_OK;
    if (!A || (total_len > 0 && (!y || !x || !dt || !B || !C)) || (max_slots > 0 && !ssm_pool))
        return SSD_ERR_INVALID_ARG;
    for (const void *q : {static_cast<const void *>(y), x, dt, B, C, z, static_cast<const void *>(A),
                          static_cast<const void *>(ssm_pool)})
        if (!kv_aligned16(q))
            return SSD_ERR_INVALID_ARG;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
        workspace_bytes < ssd_selective_scan_varlen_workspace_size(total_len, batch, channels, dstate))
        return SSD_ERR_WORKSPACE;
    p.y = static_cast<__nv_bfloat16 *>(y);
    p.x = static_cast<const __nv_bfloat16 *>(x);
    p.dt = static_cast<const __nv_bfloat16 *>(dt);
    p.B = static_cast<const __nv_bfloat16 *>(B);
    p.C = static_cast<const __nv_bfloat16 *>(C);
    p.z = static_cast<const __nv_bfloat16 *>(z);
    p.A = A;
    p.D = D;
    p.dt_bias = dt_bias;
    p.pool = ssm_pool;
    p.y_stride = t.y;
    p.x_stride = t.x;
    p.dt_stride = t.dt;
    p.b_stride = t.B;
    p.c_stride = t.C;
    p.z_stride = t.z;
    p.channels = channels;
    p.softplus = dt_softplus != 0;
    const bool bf16 = pool_type == SSD_POOL_BF16;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = dstate == 8    ? launch<8>(p, bf16, s)
                          : dstate == 16 ? launch<16>(p, bf16, s)
                          : dstate == 32 ? launch<32>(p, bf16, s)
                                         : launch<64>(p, bf16, s);
    return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
