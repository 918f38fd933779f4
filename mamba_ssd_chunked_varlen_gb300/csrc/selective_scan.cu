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
// A channel is N / 8 lanes of eight states; a warp is 256 / N channels on its own.  Tokens
// go in groups of eight, and in a group in pairs: a pair's arguments, inputs and sums are
// two fp32 each in one instruction, the states take the two one after the other.  Each of a
// channel's lanes makes the steps of its share of a group's tokens, a group ahead, and
// hands them over by shuffles; its share of the sums comes back from a reduction that
// halves the sums as it halves the lanes.  The CTA copies blocks of 16 tokens to shared
// memory two blocks ahead and lays their B and C out in fp32, a pair's two values side by
// side, so that a lane reads four operands at once.
#include <algorithm>

#include "attn_ptx.cuh"
#include "layer_common.cuh"

namespace ssd {
namespace {

constexpr int kScanWarps = 4;
constexpr int kScanThreads = kScanWarps * 32;
constexpr int kStates = 8;            // states of a lane
constexpr int kGroup = 8;             // tokens of a group
constexpr int kBlock = 16;            // tokens of a block
constexpr int kStages = 3;            // blocks in shared memory
constexpr int kShort = 7;             // tokens of a sequence that goes without shared memory

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
// max(v, 0) + log(1 + e^-|v|).  With e = e^-|v| in (0, 1], log(1 + e) = e P(e), P of degree
// 9 fitted to log(1 + e) / e (relative error 5e-9, 1.6e-7 with fp32's roundings): small
// steps keep their relative precision.
__device__ __forceinline__ float step_of(float v)
{
    const float e = ptx::ex2(-1.4426950408889634f * fabsf(v));
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

// ---------------------------------------------------------------- copies
// 16 bytes from global to shared memory without registers; zeros where there is no source.
__device__ __forceinline__ void copy16(void *dst, const void *src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(dst)), "l"(src),
                 "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// ---------------------------------------------------------------- pool
template <bool kBf16>
__device__ __forceinline__ void load_states(const void *pool, int64_t at, float (&h)[kStates])
{
    if constexpr (kBf16) {
        widen8(*reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(pool) + at), h);
    } else {
        const float4 *src = reinterpret_cast<const float4 *>(static_cast<const float *>(pool) + at);
        *reinterpret_cast<float4 *>(h) = src[0];
        *reinterpret_cast<float4 *>(h + 4) = src[1];
    }
}

template <bool kBf16>
__device__ __forceinline__ void store_states(void *pool, int64_t at, const float (&h)[kStates])
{
    if constexpr (kBf16) {
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(pool) + at) = round8(h);
    } else {
        float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(pool) + at);
        dst[0] = make_float4(h[0], h[1], h[2], h[3]);
        dst[1] = make_float4(h[4], h[5], h[6], h[7]);
    }
}

// ---------------------------------------------------------------- lanes
// Shared memory of a CTA.  Rows are padded so that the lanes of a warp that read
// several tokens at once find them in different banks.
template <int N>
struct SelShared {
    static constexpr int kLanes = N / kStates;                  // lanes of a channel
    static constexpr int kChannels = 32 / kLanes;               // channels of a warp
    static constexpr int kCols = kScanWarps * kChannels;        // of the CTA
    static constexpr int kPitch = kCols + (kLanes == 2 ? 16 : 8);
    struct Block {
        __nv_bfloat16 x[kBlock][kPitch], dt[kBlock][kPitch], z[kBlock][kPitch], B[kBlock][N], C[kBlock][N];
    };
    Block block[kStages];
    __nv_bfloat16 y[2][kBlock][kPitch];
    // per pair of tokens, [chunk][part]: two states of a part for the two tokens
    float4 B[2][kBlock / 2][kStates / 2][kLanes], C[2][kBlock / 2][kStates / 2][kLanes];
};

// What a lane holds of its channel.
struct SelLane {
    float h[kStates];
    float a[kStates];          // A log2(e)
    float D, bias;
    bool softplus;

    __device__ __forceinline__ float step(__nv_bfloat16 raw) const
    {
        const float v = __bfloat162float(raw) + bias, d = step_of(v);
        return softplus ? d : v;
    }

    // The states over a pair of tokens, whose steps are dt, inputs (before B) u; B and C of
    // the lane's states are kStride float4 apart.  Returns the pair's sums of C h.
    template <int kStride>
    __device__ __forceinline__ uint64_t pair(uint64_t dt, uint64_t u, const float4 *B, const float4 *C)
    {
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int k = 0; k < kStates / 2; ++k) {
            const float4 b = B[k * kStride], c = C[k * kStride];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float e0, e1, in0, in1;
                ptx::unpack2(ptx::mul2(dt, ptx::pack2(a[2 * k + i], a[2 * k + i])), e0, e1);
                ptx::unpack2(ptx::mul2(u, i ? ptx::pack2(b.z, b.w) : ptx::pack2(b.x, b.y)), in0, in1);
                const float first = fmaf(ptx::ex2(e0), h[2 * k + i], in0);
                h[2 * k + i] = fmaf(ptx::ex2(e1), first, in1);
                sum[i] = ptx::fma2(ptx::pack2(first, h[2 * k + i]), i ? ptx::pack2(c.z, c.w) : ptx::pack2(c.x, c.y),
                                   sum[i]);
            }
        }
        return ptx::add2(sum[0], sum[1]);
    }

    // One token, B and C of the lane's states in bf16; returns the sum of C h.
    __device__ __forceinline__ float token(float dt, float u, const uint4 &braw, const uint4 &craw)
    {
        float b[8], c[8], sum = 0.f;
        widen8(braw, b);
        widen8(craw, c);
#pragma unroll
        for (int n = 0; n < kStates; ++n) {
            h[n] = fmaf(ptx::ex2(dt * a[n]), h[n], u * b[n]);
            sum = fmaf(h[n], c[n], sum);
        }
        return sum;
    }
};

// Sums over a channel's lanes of kLanes tokens at once: lane `part` gets token part's.
template <int kLanes, int kChannels>
__device__ __forceinline__ float reduce_tokens(float *v, int part)
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

template <int N, bool kBf16, bool kGate>
__global__ void __launch_bounds__(kScanThreads) selective_scan_kernel(const __grid_constant__ SelParams p)
{
    using Shared = SelShared<N>;
    constexpr int kLanes = Shared::kLanes, kChannels = Shared::kChannels, kCols = Shared::kCols;
    constexpr int kMine = kGroup / kLanes;           // tokens of a group that a lane makes the steps of
    extern __shared__ __align__(16) uint8_t smem[];
    Shared &s = *reinterpret_cast<Shared *>(smem);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int part = lane / kChannels, in_warp = lane % kChannels, col = warp * kChannels + in_warp;
    const int b = blockIdx.x / p.tiles, col0 = blockIdx.x % p.tiles * kCols;
    const bool valid = col0 + col < p.channels;
    const int ch = valid ? col0 + col : 0;    // (the other lanes follow a channel that is there)
    pdl_wait();
    int32_t begin, end;
    if (!seq_rows(p.s.qsl, p.s.total_len, p.s.errors, b, begin, end))
        return;
    const int64_t slot = seq_slot(p.s, b);
    const bool has = slot >= 0 && p.s.has_init && p.s.has_init[b];
    const int64_t at = (slot * p.channels + ch) * N + part * kStates;

    // copies of a block's rows, 16 bytes at a time
    constexpr int kRowLoads = kCols / 8, kBcLoads = N / 8;
    auto fetch = [&](int t0) {
        typename Shared::Block &dst = s.block[(t0 - begin) / kBlock % kStages];
#pragma unroll
        for (int i0 = 0; i0 < kBlock * kRowLoads; i0 += kScanThreads) {
            const int i = i0 + threadIdx.x, row = i / kRowLoads, c = i % kRowLoads * 8;
            if (kBlock * kRowLoads % kScanThreads == 0 || i < kBlock * kRowLoads) {
                const bool there = t0 + row < end && col0 + c < p.channels;
                const int64_t t = there ? t0 + row : begin;
                const int from = there ? col0 + c : 0;
                copy16(&dst.x[row][c], p.x + t * p.x_stride + from, there);
                copy16(&dst.dt[row][c], p.dt + t * p.dt_stride + from, there);
                if constexpr (kGate)
                    copy16(&dst.z[row][c], p.z + t * p.z_stride + from, there);
            }
        }
#pragma unroll
        for (int i0 = 0; i0 < 2 * kBlock * kBcLoads; i0 += kScanThreads) {
            const int i = i0 + threadIdx.x, row = i / kBcLoads % kBlock, c = i % kBcLoads * 8;
            if (2 * kBlock * kBcLoads % kScanThreads == 0 || i < 2 * kBlock * kBcLoads) {
                const bool there = t0 + row < end, is_c = i >= kBlock * kBcLoads;
                const int64_t t = there ? t0 + row : begin;
                copy16(is_c ? &dst.C[row][c] : &dst.B[row][c],
                       (is_c ? p.C + t * p.c_stride : p.B + t * p.b_stride) + c, there);
            }
        }
        copies_commit();
    };
    const bool staged = end - begin > kShort;
    if (staged) {
        fetch(begin);
        if (begin + kBlock < end)
            fetch(begin + kBlock);
    }
    SelLane me;
#pragma unroll
    for (int n = 0; n < kStates; ++n)
        me.h[n] = 0.f;
    if (has)
        load_states<kBf16>(p.pool, at, me.h);
#pragma unroll
    for (int n = 0; n < kStates; n += 4) {
        const float4 v = __ldg(reinterpret_cast<const float4 *>(p.A + static_cast<int64_t>(ch) * N + part * kStates + n));
        me.a[n] = v.x * 1.4426950408889634f;
        me.a[n + 1] = v.y * 1.4426950408889634f;
        me.a[n + 2] = v.z * 1.4426950408889634f;
        me.a[n + 3] = v.w * 1.4426950408889634f;
    }
    me.D = p.D ? p.D[ch] : 0.f;
    me.bias = p.dt_bias ? p.dt_bias[ch] : 0.f;
    me.softplus = p.softplus;
    auto output = [&](float sum, float x, __nv_bfloat16 z) {
        float v = fmaf(me.D, x, sum);
        if constexpr (kGate)
            v *= silu_f32(__bfloat162float(z));
        return __float2bfloat16_rn(v);
    };
    const __nv_bfloat16 none = __float2bfloat16_rn(0.f);

    if (!staged) {
        // a few tokens: straight from global memory
        for (int t = begin; t < end; ++t) {
            const __nv_bfloat16 z = kGate ? p.z[t * p.z_stride + ch] : none;
            const float x = __bfloat162float(p.x[t * p.x_stride + ch]), dt = me.step(p.dt[t * p.dt_stride + ch]);
            float sum = me.token(dt, dt * x,
                                 *reinterpret_cast<const uint4 *>(p.B + t * p.b_stride + part * kStates),
                                 *reinterpret_cast<const uint4 *>(p.C + t * p.c_stride + part * kStates));
#pragma unroll
            for (int o = kChannels; o < 32; o <<= 1)
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (part == 0 && valid)
                p.y[t * p.y_stride + ch] = output(sum, x, z);
        }
        if (slot >= 0 && valid)
            store_states<kBf16>(p.pool, at, me.h);
        return;
    }

    // B and C of a block in fp32, pair by pair
    auto lay_out = [&](int k) {
        const typename Shared::Block &src = s.block[k % kStages];
        constexpr int kItems = kBlock / 2 * (N / 2);
#pragma unroll
        for (int i0 = 0; i0 < kItems; i0 += kScanThreads) {
            const int i = i0 + threadIdx.x;
            if (kItems % kScanThreads == 0 || i < kItems) {
                const int pair = i / (N / 2), n = i % (N / 2) * 2, to_part = n / kStates, chunk = n % kStates / 2;
                auto two = [&](const __nv_bfloat16 (*v)[N]) {
                    const uint32_t t0 = *reinterpret_cast<const uint32_t *>(&v[2 * pair][n]);
                    const uint32_t t1 = *reinterpret_cast<const uint32_t *>(&v[2 * pair + 1][n]);
                    return make_float4(__uint_as_float(t0 << 16), __uint_as_float(t1 << 16),
                                       __uint_as_float(t0 & 0xffff0000u), __uint_as_float(t1 & 0xffff0000u));
                };
                s.B[k & 1][pair][chunk][to_part] = two(src.B);
                s.C[k & 1][pair][chunk][to_part] = two(src.C);
            }
        }
    };
    // y of block k from shared memory, 16 bytes at a time
    auto write_out = [&](int k) {
        const int t0 = begin + k * kBlock;
#pragma unroll
        for (int i0 = 0; i0 < kBlock * kRowLoads; i0 += kScanThreads) {
            const int i = i0 + threadIdx.x, row = i / kRowLoads, c = i % kRowLoads * 8;
            if ((kBlock * kRowLoads % kScanThreads == 0 || i < kBlock * kRowLoads) && t0 + row < end &&
                col0 + c < p.channels)
                *reinterpret_cast<uint4 *>(p.y + (t0 + row) * p.y_stride + col0 + c) =
                    *reinterpret_cast<const uint4 *>(&s.y[k & 1][row][c]);
        }
    };
    // the steps of the lane's tokens of a group
    float dt[kMine], u[kMine], x[kMine];
    __nv_bfloat16 z[kMine];
    auto steps = [&](const typename Shared::Block &src, int row0, float (&dt)[kMine], float (&u)[kMine],
                     float (&x)[kMine], __nv_bfloat16 (&z)[kMine]) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int row = row0 + i * kLanes + part;
            x[i] = __bfloat162float(src.x[row][col]);
            z[i] = kGate ? src.z[row][col] : none;
            dt[i] = me.step(src.dt[row][col]);
            u[i] = dt[i] * x[i];
        }
    };

    copies_wait();
    __syncthreads();
    lay_out(0);
    steps(s.block[0], 0, dt, u, x, z);
    const int blocks = (end - begin + kBlock - 1) / kBlock;
    for (int k = 0; k < blocks; ++k) {
        // block k + 1 has arrived for everybody, and nobody reads blocks and y of k - 1 any more
        copies_wait();
        __syncthreads();
        const int t0 = begin + k * kBlock, n = min(kBlock, end - t0);
        if (t0 + 2 * kBlock < end)
            fetch(t0 + 2 * kBlock);
        if (k > 0)
            write_out(k - 1);
        if (k + 1 < blocks)
            lay_out(k + 1);
        const typename Shared::Block &now = s.block[k % kStages], &next = s.block[(k + 1) % kStages];
        int g = 0;
        for (; g + kGroup <= n; g += kGroup) {
            // the next group's steps go between this one's (past the end they are not used)
            float dt1[kMine], u1[kMine], x1[kMine];
            __nv_bfloat16 z1[kMine];
            const bool more = g + kGroup < kBlock;
            steps(more ? now : next, more ? g + kGroup : 0, dt1, u1, x1, z1);
            float sums[kGroup];
#pragma unroll
            for (int j = 0; j < kGroup; j += 2) {
                uint64_t dt2, u2;
                if constexpr (kLanes == 1) {
                    dt2 = ptx::pack2(dt[j], dt[j + 1]);
                    u2 = ptx::pack2(u[j], u[j + 1]);
                } else {
                    const int i = j / kLanes, from = j % kLanes * kChannels + in_warp;
                    dt2 = ptx::pack2(__shfl_sync(0xffffffffu, dt[i], from),
                                     __shfl_sync(0xffffffffu, dt[i], from + kChannels));
                    u2 = ptx::pack2(__shfl_sync(0xffffffffu, u[i], from),
                                    __shfl_sync(0xffffffffu, u[i], from + kChannels));
                }
                const int row = (g + j) / 2;
                ptx::unpack2(me.pair<kLanes>(dt2, u2, &s.B[k & 1][row][0][part], &s.C[k & 1][row][0][part]), sums[j],
                             sums[j + 1]);
            }
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                const float sum = reduce_tokens<kLanes, kChannels>(sums + i * kLanes, part);
                s.y[k & 1][g + i * kLanes + part][col] = output(sum, x[i], z[i]);
            }
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                dt[i] = dt1[i];
                u[i] = u1[i];
                x[i] = x1[i];
                z[i] = z1[i];
            }
        }
        for (; g < n; ++g) {      // the sequence's last tokens, fewer than a group
            const float xt = __bfloat162float(now.x[g][col]), d = me.step(now.dt[g][col]);
            float sum = me.token(d, d * xt, *reinterpret_cast<const uint4 *>(&now.B[g][part * kStates]),
                                 *reinterpret_cast<const uint4 *>(&now.C[g][part * kStates]));
#pragma unroll
            for (int o = kChannels; o < 32; o <<= 1)
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (part == 0)
                s.y[k & 1][g][col] = output(sum, xt, kGate ? now.z[g][col] : none);
        }
    }
    __syncthreads();
    write_out(blocks - 1);
    if (slot >= 0 && valid)
        store_states<kBf16>(p.pool, at, me.h);
}

template <int N, bool kBf16, bool kGate>
cudaError_t launch(SelParams &p, cudaStream_t stream)
{
    using Shared = SelShared<N>;
    constexpr int kBytes = sizeof(Shared);
    cudaError_t e = cudaFuncSetAttribute(selective_scan_kernel<N, kBf16, kGate>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e != cudaSuccess)
        return e;
    p.tiles = (p.channels + Shared::kCols - 1) / Shared::kCols;
    return launch_pdl_smem(selective_scan_kernel<N, kBf16, kGate>, dim3(static_cast<unsigned>(p.tiles * p.s.batch)),
                           kScanThreads, kBytes, stream, p);
}

template <int N>
cudaError_t launch(SelParams &p, bool bf16, cudaStream_t stream)
{
    if (p.z)
        return bf16 ? launch<N, true, true>(p, stream) : launch<N, false, true>(p, stream);
    return bf16 ? launch<N, true, false>(p, stream) : launch<N, false, false>(p, stream);
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
