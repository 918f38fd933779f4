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
// go in pairs: a pair's arguments, inputs and sums are two fp32 each in one instruction,
// the states take the two one after the other.  Each of a channel's lanes makes the
// steps of its share of a group's pairs, a group ahead and two at a time as well, and hands
// them over through shared memory; its share of the sums comes back from a reduction that
// halves the sums as it halves the lanes.  The CTA copies blocks of 16 or 32 tokens to
// shared memory two or three blocks ahead and lays their B and C out in fp32, a pair's two
// values side by side, so that a lane reads four operands at once.
//
// A sequence that would keep too few warps busy is cut into chunks (sel_chunk).  A first
// kernel does the first chunks, and makes the states alone that each further one but the last
// leads to from zero, and the sums of their steps; in the second a chunk joins what lies
// before it, h = exp(A sum dt) h + the next chunk's own, and does its tokens.  (With the first
// chunks in the second kernel, too, and smallest chunks of 64: 20 single tokens and 4 of 427 on
// average, 4,096 channels 63 us instead of 62, one of 9,763 and 8,192, cut then, 565 and 532.)  One
// CTA lists the chunks before, the long ones first.  Batches of single tokens, whose work is to
// read and write the states, go to a kernel whose CTAs keep their tile's decays and have
// the next sequences' states on their way.
#include <algorithm>
#include <type_traits>

#include "attn_ptx.cuh"
#include "kernels.cuh"
#include "layer_common.cuh"

namespace ssd {
namespace {

constexpr int kScanWarps = 4;
constexpr int kScanThreads = kScanWarps * 32;
constexpr int kChunkStep = 16;        // chunks are multiples of so many tokens
constexpr int kFew = 8;               // tokens of a sequence that goes without shared memory

constexpr int kStates = 8;            // states of a lane
constexpr int kMinChunk = 48;         // tokens of a chunk at least
constexpr int kFullWarps = 5000;      // warps that sel_chunk wants of a call's chunks
constexpr int kResident = 4;          // CTAs of an SM at most

// A chunk k of a sequence, as a rule the whole sequence.
struct alignas(32) SelUnit {
    int32_t seq, begin, end;          // its tokens [begin, end)
    int32_t k, ends;                  // index; where the ends of the sequence's chunks begin
    int32_t cut, last, pad;           // whether the sequence is cut, whether it is its last
};

struct SelHeader {
    int32_t units, ends;              // chunks; of them not the last of their sequence
};

struct SelParams {
    SlotBatch s;
    __nv_bfloat16 *y;
    const __nv_bfloat16 *x, *dt, *B, *C, *z;
    const float *A, *D, *dt_bias;
    void *pool;
    SelHeader *header;
    SelUnit *units, *later;           // whole sequences and chunks with an end, long ones first (null:
                                      // all are whole, in order); the chunk behind each end
    float *ends, *sums;               // [end]: states and steps' sum of the chunk before it
    int32_t y_stride, x_stride, dt_stride, b_stride, c_stride, z_stride;
    int32_t channels, tiles;          // tiles of a CTA's channels
    int32_t chunk, warps;             // smallest chunk (0: nothing is cut), warps of a sequence
    int32_t few;                      // tokens of the sequences that the kernel of few takes
    int32_t softplus, pool_bf16;
    int32_t behind;                   // `units` are the chunks behind ends
};

// ---------------------------------------------------------------- chunks
// Warps of a sequence, and tokens of the smallest chunk: as many as give kFullWarps warps
// over all tokens.
inline int64_t sel_warps(int32_t channels, int32_t dstate)
{
    return (static_cast<int64_t>(channels) * dstate + 32 * kStates - 1) / (32 * kStates);
}
inline int32_t sel_chunk(int64_t total_len, int32_t channels, int32_t dstate)
{
    const int64_t tokens = (total_len * sel_warps(channels, dstate) + kFullWarps - 1) / kFullWarps;
    const int64_t steps = (tokens + kChunkStep - 1) / kChunkStep;
    return static_cast<int32_t>(std::min<int64_t>(std::max<int64_t>(kMinChunk, steps * kChunkStep), INT32_MAX / 2));
}

// What a call takes, in ns, whose sequences of some length on are cut: its longest whole
// sequence, or all of its tokens.  Measured, of 16 states: a token of a whole sequence 64 up to 4,096
// channels, 90 of 8,192, taken as 80; a token and warp of a whole sequence 0.086, of a cut one (most
// of whose states are made twice) 0.115; the additional kernel 6,000.  (Whole and cut, one
// sequence of 4,096 tokens, 2,048 channels: 263 and 79 us; of 500 tokens, 4,096 channels: 38 and 27.)
__device__ __forceinline__ float sel_cost(int longest, int whole, int cut, int warps)
{
    return fmaxf(80.f * longest, (0.086f * whole + 0.115f * cut) * warps) + (cut > 0 ? 6000.f : 0.f);
}

// Lists the chunks of the sequences of more than p.few tokens: `count` of `len` tokens a
// sequence, the last one shorter.  Which lengths are cut is up to sel_cost, by powers of two.
constexpr int kPlanThreads = 512;
constexpr int kPlanSizes = 30;        // powers of two: all that a sequence's length can have

__device__ __forceinline__ int sel_size(int32_t len) { return 31 - __clz(len | 1); }

__global__ void __launch_bounds__(kPlanThreads) selective_plan_kernel(const __grid_constant__ SelParams p)
{
    __shared__ int s_units[kPlanSizes], s_tokens[kPlanSizes], s_longest[kPlanSizes], s_ends, s_cut;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x < kPlanSizes) {
        s_units[threadIdx.x] = 0;
        s_tokens[threadIdx.x] = 0;
        s_longest[threadIdx.x] = 0;
    }
    if (threadIdx.x == 0) {
        s_ends = 0;
        s_cut = INT32_MAX;
    }
    pdl_wait();
    __syncthreads();
    // the thread's first sequence stays in registers, as a rule there are no others
    int32_t begin0 = 0, end0 = -1;
    if (threadIdx.x < p.s.batch && !seq_rows(p.s.qsl, p.s.total_len, p.s.errors, threadIdx.x, begin0, end0))
        end0 = -1;
    auto rows = [&](int b, int32_t &begin, int32_t &end) {
        begin = begin0;
        end = end0;
        return b < kPlanThreads ? end0 >= 0
                                : b < p.s.batch && seq_rows(p.s.qsl, p.s.total_len, p.s.errors, b, begin, end);
    };
    int32_t begin, end, len = 0;
    if (p.chunk) {
        bool bad = false;
        for (int b = threadIdx.x; b < p.s.batch; b += kPlanThreads) {
            if (!rows(b, begin, end)) {
                bad = true;
                continue;
            }
            if (end - begin <= p.few)
                continue;
            atomicAdd(&s_tokens[sel_size(end - begin)], end - begin);
            atomicMax(&s_longest[sel_size(end - begin)], end - begin);
        }
        // (with offsets that fall, the sequences may come to more than the workspace is for)
        if (!__syncthreads_or(bad) && threadIdx.x < 32) {
            // a lane is a size; what a call takes with all from that size on cut
            const int tokens = lane < kPlanSizes ? s_tokens[lane] : 0;
            int upto = warp_inclusive_scan(tokens), longest = lane < kPlanSizes ? s_longest[lane] : 0;
            const int all = __shfl_sync(0xffffffffu, upto, 31);
#pragma unroll
            for (int o = 1; o < kPlanSizes; o <<= 1) {
                const int other = __shfl_up_sync(0xffffffffu, longest, o);
                longest = max(longest, lane >= o ? other : 0);
            }
            const float whole = sel_cost(__shfl_sync(0xffffffffu, longest, kPlanSizes - 1), all, 0, p.warps);
            int below = __shfl_up_sync(0xffffffffu, longest, 1);
            below = lane > 0 ? below : 0;
            upto -= tokens;
            float best = lane < kPlanSizes && 1 << lane > p.chunk ? sel_cost(below, upto, all - upto, p.warps) : whole;
            int size = lane;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const float cost = __shfl_xor_sync(0xffffffffu, best, o);
                const int other = __shfl_xor_sync(0xffffffffu, size, o);
                if (cost < best || (cost == best && other > size)) {
                    best = cost;
                    size = other;
                }
            }
            if (lane == 0 && best < whole)
                s_cut = max(1 << size, 2 * p.chunk);
        }
        __syncthreads();
    }
    const int32_t shortest = s_cut;
    auto chunks = [&](int b, int &count) {
        count = 0;
        if (!rows(b, begin, end) || end - begin <= p.few)
            return 0;
        len = end - begin;
        count = 1;
        if (len >= shortest) {
            const int32_t n = len / p.chunk;
            len = ((len + n - 1) / n + kChunkStep - 1) / kChunkStep * kChunkStep;
            count = (end - begin + len - 1) / len;
        }
        return kPlanSizes - 1 - sel_size(len);      // long ones first
    };
    int count;
    for (int b = threadIdx.x; b < p.s.batch; b += kPlanThreads) {
        const int size = chunks(b, count);
        if (count)
            atomicAdd(&s_units[size], max(1, count - 1));
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const int n = lane < kPlanSizes ? s_units[lane] : 0, upto = warp_inclusive_scan(n);
        if (lane < kPlanSizes)
            s_units[lane] = upto - n;
        if (lane == 31)
            p.header->units = upto;
    }
    __syncthreads();
    for (int b0 = threadIdx.x - lane; b0 < p.s.batch; b0 += kPlanThreads) {
        const int b = b0 + lane, size = chunks(b, count);
        int at = 0, ends = 0;
        if (count) {
            at = atomicAdd(&s_units[size], max(1, count - 1));
            if (count > 1)
                ends = atomicAdd(&s_ends, count - 1);
            else
                p.units[at] = SelUnit{b, begin, end, 0, 0, 0, 1, 0};
        }
        for (uint32_t many = __ballot_sync(0xffffffffu, count > 1); many; many &= many - 1) {
            const int from = __ffs(many) - 1;
            const int n = __shfl_sync(0xffffffffu, count, from), first = __shfl_sync(0xffffffffu, begin, from);
            const int behind = __shfl_sync(0xffffffffu, end, from), l = __shfl_sync(0xffffffffu, len, from);
            const int u = __shfl_sync(0xffffffffu, at, from), e = __shfl_sync(0xffffffffu, ends, from);
            for (int k = lane; k < n; k += 32) {
                const SelUnit unit = {b0 + from, first + k * l, min(first + (k + 1) * l, behind), k, e, 1, k == n - 1, 0};
                if (k < n - 1)
                    p.units[u + k] = unit;
                if (k > 0)
                    p.later[e + k - 1] = unit;
            }
        }
    }
    __syncthreads();
    if (threadIdx.x == 0)
        p.header->ends = s_ends;
}

// ---------------------------------------------------------------- arithmetic
// A value twice.  (Volatile: made once and kept, not again at each use.)
__device__ __forceinline__ uint64_t twice(float v)
{
    uint64_t r;
    asm volatile("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(v));
    return r;
}

// log(1 + e) / e on [0, 1] by the polynomial of degree 8 whose largest relative error is smallest (by
// Remez's exchange: 3.0e-8).  With its coefficients in fp32 6.4e-8, the last one's rounding for small
// e; with fp32's operations log(1 + e) is off by 1.8e-7.
#define SSD_LOG1P_TERMS(F) \
    F(0.0052326940931379795f) F(-0.029505237936973572f) F(0.07822595536708832f) F(-0.13663245737552643f) \
    F(0.19106006622314453f) F(-0.2484298199415207f) F(0.3331909775733948f) F(-0.4999949336051941f) \
    F(0.9999999403953552f)

constexpr float kLog2e = 1.4426950408889634f;

// softplus(v) = max(v, 0) + log(1 + e) with e = e^-|v| in (0, 1]: small steps keep their
// relative precision.
__device__ __forceinline__ float step_of(float v)
{
    const float e = ptx::ex2(-fabsf(v * kLog2e));
    float p = 0.f;
#define SSD_TERM(c) p = fmaf(p, e, c);
    SSD_LOG1P_TERMS(SSD_TERM)
#undef SSD_TERM
    return fmaf(p, e, fmaxf(v, 0.f));
}

// What two tokens' steps and outputs need, each value twice.
struct Pairwise {
    uint64_t terms[9], log2e, bias, D;
    bool softplus;

    __device__ __forceinline__ void set(float bias_, float D_, bool softplus_)
    {
        int i = 0;
#define SSD_TERM(c) terms[i++] = twice(c);
        SSD_LOG1P_TERMS(SSD_TERM)
#undef SSD_TERM
        log2e = twice(kLog2e);
        bias = twice(bias_);
        D = twice(D_);
        softplus = softplus_;
    }

    // steps of two raw values: step_of on each
    __device__ __forceinline__ uint64_t steps(float raw0, float raw1) const
    {
        const uint64_t v = ptx::add2(ptx::pack2(raw0, raw1), bias);
        float v0, v1, t0, t1, d0, d1;
        ptx::unpack2(v, v0, v1);
        ptx::unpack2(ptx::mul2(v, log2e), t0, t1);
        const uint64_t e = ptx::pack2(ptx::ex2(-fabsf(t0)), ptx::ex2(-fabsf(t1)));
        uint64_t p = ptx::fma2(terms[0], e, terms[1]);
#pragma unroll
        for (int i = 2; i < 9; ++i)
            p = ptx::fma2(p, e, terms[i]);
        ptx::unpack2(ptx::fma2(p, e, ptx::pack2(fmaxf(v0, 0.f), fmaxf(v1, 0.f))), d0, d1);
        return ptx::pack2(softplus ? d0 : v0, softplus ? d1 : v1);
    }

    // two outputs of sums of C h, x and the gate
    template <bool kGate>
    __device__ __forceinline__ uint32_t outputs(uint64_t sum, uint64_t x, float z0, float z1) const
    {
        uint64_t v = ptx::fma2(D, x, sum);
        if constexpr (kGate) {
            float t0, t1, q0, q1;
            ptx::unpack2(ptx::mul2(ptx::pack2(z0, z1), log2e), t0, t1);
            ptx::unpack2(ptx::add2(ptx::pack2(ptx::ex2(-t0), ptx::ex2(-t1)), ptx::pack2(1.f, 1.f)), q0, q1);
            v = ptx::mul2(ptx::mul2(v, ptx::pack2(z0, z1)), ptx::pack2(rcp_f32(q0), rcp_f32(q1)));
        }
        float v0, v1;
        ptx::unpack2(v, v0, v1);
        return pack_bf16(v0, v1);
    }
};

// ---------------------------------------------------------------- copies
// 16 bytes from global to shared memory without registers; zeros where there is no source.
__device__ __forceinline__ void copy16(void *dst, const void *src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(dst)), "l"(src),
                 "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until all but the last kBehind groups of copies have arrived.
template <int kBehind>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(kBehind) : "memory");
}

// ---------------------------------------------------------------- states
__device__ __forceinline__ void load_bf16(const __nv_bfloat16 *src, float (&v)[kStates])
{
    widen8(*reinterpret_cast<const uint4 *>(src), v);
}

// A lane's states from the pool and into it.
__device__ __forceinline__ void load_states(const void *pool, bool bf16, int64_t at, float (&h)[kStates])
{
    if (bf16) {
        load_bf16(static_cast<const __nv_bfloat16 *>(pool) + at, h);
        return;
    }
#pragma unroll
    for (int i = 0; i < kStates; i += 4) {
        const float4 v = *reinterpret_cast<const float4 *>(static_cast<const float *>(pool) + at + i);
        h[i] = v.x;
        h[i + 1] = v.y;
        h[i + 2] = v.z;
        h[i + 3] = v.w;
    }
}

__device__ __forceinline__ void store_states(void *pool, bool bf16, int64_t at, const float (&h)[kStates])
{
#pragma unroll
    for (int i = 0; i < kStates; i += 4) {
        if (bf16)
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(pool) + at + i) =
                make_uint2(pack_bf16(h[i], h[i + 1]), pack_bf16(h[i + 2], h[i + 3]));
        else
            *reinterpret_cast<float4 *>(static_cast<float *>(pool) + at + i) =
                make_float4(h[i], h[i + 1], h[i + 2], h[i + 3]);
    }
}

// ---------------------------------------------------------------- lanes
// Shared memory of a CTA.  Rows are padded so that the lanes of a warp that read
// several tokens at once find them in different banks.
template <int N, int kBlock>
struct SelShared {
    static constexpr int kStages = kBlock == 16 ? 4 : 3;        // blocks
    static constexpr int kLanes = N / kStates;                  // lanes of a channel
    static constexpr int kChannels = 32 / kLanes;               // channels of a warp
    static constexpr int kCols = kScanWarps * kChannels;        // of the CTA
    static constexpr int kPitch = kCols + (kLanes == 2 ? 16 : 8);
    struct Block {
        __nv_bfloat16 x[kBlock][kPitch], dt[kBlock][kPitch], z[kBlock][kPitch], B[kBlock][N], C[kBlock][N];
    };
    Block block[kStages];
    __nv_bfloat16 y[2][kBlock][kPitch];
    // per warp, two groups: the steps and the inputs before B of a pair {d0, d1, u0, u1}
    static constexpr int kGroup = kLanes == 8 || kBlock == 32 ? 16 : 8;              // tokens of a group
    float4 steps[2][kScanWarps][kGroup / 2][kChannels];
    // per pair of tokens, [chunk][part]: two states of a part for the two tokens
    float4 B[2][kBlock / 2][kStates / 2][kLanes], C[2][kBlock / 2][kStates / 2][kLanes];
};

// CTAs of an SM that have room for it, at most `most`.
template <int N, int kBlock>
constexpr int sel_resident(int most)
{
    const int room = (kMaxSmemPerBlock + 1024) / static_cast<int>(sizeof(SelShared<N, kBlock>) + 1024);
    return room < most ? room : most;
}

// What a lane holds of its channel.
struct SelLane {
    float h[kStates];
    uint64_t a[kStates];       // A log2(e), twice

    __device__ __forceinline__ void load_decays(const float *A)
    {
#pragma unroll
        for (int n = 0; n < kStates; n += 4) {
            const float4 v = __ldg(reinterpret_cast<const float4 *>(A + n));
            a[n] = twice(v.x * kLog2e);
            a[n + 1] = twice(v.y * kLog2e);
            a[n + 2] = twice(v.z * kLog2e);
            a[n + 3] = twice(v.w * kLog2e);
        }
    }
    __device__ __forceinline__ float decay(int n) const
    {
        float v, same;
        ptx::unpack2(a[n], v, same);
        return v;
    }

    // The states over a pair of tokens, whose steps are dt, inputs (before B) u; B and C of
    // the lane's states are kStride float4 apart.  Returns the pair's sums of C h (kOut).
    template <int kStride, bool kOut>
    __device__ __forceinline__ uint64_t pair(uint64_t dt, uint64_t u, const float4 *B, const float4 *C)
    {
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int k = 0; k < kStates / 2; ++k) {
            const float4 b = B[k * kStride], c = kOut ? C[k * kStride] : make_float4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float e0, e1, in0, in1;
                ptx::unpack2(ptx::mul2(dt, a[2 * k + i]), e0, e1);
                ptx::unpack2(ptx::mul2(u, i ? ptx::pack2(b.z, b.w) : ptx::pack2(b.x, b.y)), in0, in1);
                const float first = fmaf(ptx::ex2(e0), h[2 * k + i], in0);
                h[2 * k + i] = fmaf(ptx::ex2(e1), first, in1);
                if constexpr (kOut)
                    sum[i] = ptx::fma2(ptx::pack2(first, h[2 * k + i]),
                                       i ? ptx::pack2(c.z, c.w) : ptx::pack2(c.x, c.y), sum[i]);
            }
        }
        return ptx::add2(sum[0], sum[1]);
    }

    // One token, B and C of the lane's states in bf16; returns the sum of C h.
    __device__ __forceinline__ float token(float dt, float u, const uint4 &B, const uint4 &C)
    {
        float b[kStates], c[kStates], sum = 0.f;
        widen8(B, b);
        widen8(C, c);
#pragma unroll
        for (int n = 0; n < kStates; ++n) {
            h[n] = fmaf(ptx::ex2(dt * decay(n)), h[n], u * b[n]);
            sum = fmaf(h[n], c[n], sum);
        }
        return sum;
    }
    __device__ __forceinline__ float token(float dt, float u, const __nv_bfloat16 *B, const __nv_bfloat16 *C)
    {
        return token(dt, u, *reinterpret_cast<const uint4 *>(B), *reinterpret_cast<const uint4 *>(C));
    }
};

// Sums over a channel's lanes of kLanes pairs at once: lane `part` gets pair part's.
template <int kLanes, int kChannels>
__device__ __forceinline__ uint64_t reduce_pairs(uint64_t *v, int part)
{
#pragma unroll
    for (int n = kLanes / 2; n >= 1; n /= 2) {
        const bool upper = part & n;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const uint64_t send = upper ? v[i] : v[i + n], keep = upper ? v[i + n] : v[i];
            float s0, s1;
            ptx::unpack2(send, s0, s1);
            v[i] = ptx::add2(keep, ptx::pack2(__shfl_xor_sync(0xffffffffu, s0, n * kChannels),
                                              __shfl_xor_sync(0xffffffffu, s1, n * kChannels)));
        }
    }
    return v[0];
}

// Tokens [begin, end) of one sequence by a CTA: the lane's states over them and, with
// kOut, their y; else the sum of the channel's steps in `total`.
template <int N, bool kGate, bool kOut, int kBlock>
__device__ __forceinline__ void sel_tokens(const SelParams &p, SelShared<N, kBlock> &s, SelLane &me, int begin, int end,
                                           int col0, float D, float bias, float &total)
{
    using Shared = SelShared<N, kBlock>;
    constexpr int kLanes = Shared::kLanes, kChannels = Shared::kChannels, kCols = Shared::kCols;
    constexpr int kGroup = Shared::kGroup, kGroups = kBlock / kGroup, kStages = Shared::kStages;
    static_assert(kGroups == 1 || kGroups % 2 == 0);
    constexpr int kMine = kGroup / 2 / kLanes;       // pairs of a group that a lane makes the steps of
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int part = lane / kChannels, in_warp = lane % kChannels, col = warp * kChannels + in_warp;

    // copies of a block's rows, 16 bytes at a time
    constexpr int kRowLoads = kCols / 8, kBcLoads = N / 8, kBc = kOut ? 2 : 1;
    auto fetch = [&](int t0) {
        if (t0 >= end) {      // (groups are counted)
            copies_commit();
            return;
        }
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
                if constexpr (kGate && kOut)
                    copy16(&dst.z[row][c], p.z + t * p.z_stride + from, there);
            }
        }
#pragma unroll
        for (int i0 = 0; i0 < kBc * kBlock * kBcLoads; i0 += kScanThreads) {
            const int i = i0 + threadIdx.x, row = i / kBcLoads % kBlock, c = i % kBcLoads * 8;
            if (kBc * kBlock * kBcLoads % kScanThreads == 0 || i < kBc * kBlock * kBcLoads) {
                const bool there = t0 + row < end, is_c = i >= kBlock * kBcLoads;
                const int64_t t = there ? t0 + row : begin;
                copy16(is_c ? &dst.C[row][c] : &dst.B[row][c],
                       (is_c ? p.C + t * p.c_stride : p.B + t * p.b_stride) + c, there);
            }
        }
        copies_commit();
    };
#pragma unroll
    for (int k = 0; k + 1 < kStages; ++k)
        fetch(begin + k * kBlock);
    // one token's step and output
    auto step = [&](__nv_bfloat16 raw) {
        const float v = __bfloat162float(raw) + bias;
        return p.softplus ? step_of(v) : v;
    };
    auto output = [&](float sum, float x, __nv_bfloat16 z) {
        float v = fmaf(D, x, sum);
        if constexpr (kGate)
            v *= silu_f32(__bfloat162float(z));
        return __float2bfloat16_rn(v);
    };
    const __nv_bfloat16 none = __float2bfloat16_rn(0.f);

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
                if constexpr (kOut)
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
                *reinterpret_cast<uint4 *>(p.y + static_cast<int64_t>(t0 + row) * p.y_stride + col0 + c) =
                    *reinterpret_cast<const uint4 *>(&s.y[k & 1][row][c]);
        }
    };
    // The lane's pairs of a group: tokens 2 (i kLanes + part) and the next of it.  Their steps
    // go to the warp's shared memory, their x and z stay.
    Pairwise two;
    two.set(bias, D, p.softplus);
    struct Kept {
        uint64_t x[kMine];
        float z[kGate && kOut ? 2 * kMine : 1];
    };
    auto make_steps = [&](const typename Shared::Block &src, int row0, float4 (&made)[kMine], Kept &keep) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int pair = i * kLanes + part, row = row0 + 2 * pair;
            keep.x[i] = ptx::pack2(__bfloat162float(src.x[row][col]), __bfloat162float(src.x[row + 1][col]));
            if constexpr (kGate && kOut) {
                keep.z[2 * i] = __bfloat162float(src.z[row][col]);
                keep.z[2 * i + 1] = __bfloat162float(src.z[row + 1][col]);
            }
            const uint64_t d = two.steps(__bfloat162float(src.dt[row][col]), __bfloat162float(src.dt[row + 1][col]));
            float d0, d1, u0, u1;
            ptx::unpack2(d, d0, d1);
            ptx::unpack2(ptx::mul2(d, keep.x[i]), u0, u1);
            made[i] = make_float4(d0, d1, u0, u1);
        }
    };
    auto hand_over = [&](const float4 (&made)[kMine], float4 (&dst)[kGroup / 2][kChannels]) {
#pragma unroll
        for (int i = 0; i < kMine; ++i)
            dst[i * kLanes + part][in_warp] = made[i];
    };
    // A group from row g of block k: its states and sums, and the y of the lane's pairs.
    auto group = [&](int k, int g, const float4 (&src)[kGroup / 2][kChannels], const Kept &keep) {
        uint32_t out[kMine];
        uint64_t steps = 0;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            uint64_t sums[kLanes];
#pragma unroll
            for (int j = 0; j < kLanes; ++j) {
                const int pair = i * kLanes + j, row = g / 2 + pair;
                const float4 st = src[pair][in_warp];
                sums[j] = me.template pair<kLanes, kOut>(ptx::pack2(st.x, st.y), ptx::pack2(st.z, st.w),
                                                         &s.B[k & 1][row][0][part], &s.C[k & 1][row][0][part]);
                if constexpr (!kOut)
                    steps = ptx::add2(steps, ptx::pack2(st.x, st.y));
            }
            if constexpr (kOut)
                out[i] = two.template outputs<kGate>(reduce_pairs<kLanes, kChannels>(sums, part), keep.x[i],
                                                     keep.z[kGate ? 2 * i : 0], keep.z[kGate ? 2 * i + 1 : 0]);
        }
        if constexpr (kOut) {
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                const int row = g + 2 * (i * kLanes + part);
                s.y[k & 1][row][col] = __ushort_as_bfloat16(static_cast<unsigned short>(out[i]));
                s.y[k & 1][row + 1][col] = __ushort_as_bfloat16(static_cast<unsigned short>(out[i] >> 16));
            }
        } else {
            float d0, d1;
            ptx::unpack2(steps, d0, d1);
            total += d0 + d1;
        }
    };

    copies_wait<kStages - 2>();
    __syncthreads();
    lay_out(0);
    Kept keep[2];
    float4 made[kMine];
    make_steps(s.block[0], 0, made, keep[0]);
    hand_over(made, s.steps[0][warp]);
    const int blocks = (end - begin + kBlock - 1) / kBlock;
    for (int k = 0; k < blocks; ++k) {
        // block k + 1 has arrived for everybody, and nobody reads blocks and y of k - 1 any more
        copies_wait<kStages - 3>();
        __syncthreads();
        const int t0 = begin + k * kBlock, n = min(kBlock, end - t0);
        fetch(t0 + (kStages - 1) * kBlock);
        if (kOut && k > 0)
            write_out(k - 1);
        if (k + 1 < blocks)
            lay_out(k + 1);
        const typename Shared::Block &now = s.block[k % kStages], &next = s.block[(k + 1) % kStages];
        if (n == kBlock) {
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                // the next group's steps are made among this one's states, and stored behind
                // them, where no load has to wait for them (past the end they are not used)
                const int from = (kGroups == 1 ? k : i) & 1;
                make_steps(i + 1 < kGroups ? now : next, (i + 1) % kGroups * kGroup, made,
                           keep[kGroups == 1 ? 1 : (i + 1) & 1]);
                group(k, i * kGroup, s.steps[from][warp], keep[kGroups == 1 ? 0 : i & 1]);
                hand_over(made, s.steps[from ^ 1][warp]);
                if constexpr (kGroups == 1)
                    keep[0] = keep[1];
                __syncwarp();
            }
            continue;
        }
        int g = 0;
        if constexpr (kGroups > 1)
            for (int from = 0; g + kGroup <= n; g += kGroup, from ^= 1) {
                make_steps(now, g + kGroup, made, keep[1]);
                group(k, g, s.steps[from][warp], keep[0]);
                hand_over(made, s.steps[from ^ 1][warp]);
                keep[0] = keep[1];
                __syncwarp();
            }
        for (; g < n; ++g) {      // the sequence's last tokens, fewer than a group
            const float xt = __bfloat162float(now.x[g][col]), d = step(now.dt[g][col]);
            float sum = me.token(d, d * xt, &now.B[g][part * kStates], &now.C[g][part * kStates]);
            if constexpr (kOut) {
#pragma unroll
                for (int o = kChannels; o < 32; o <<= 1)
                    sum += __shfl_xor_sync(0xffffffffu, sum, o);
                if (part == 0)
                    s.y[k & 1][g][col] = output(sum, xt, kGate ? now.z[g][col] : none);
            } else {
                total += d;
            }
        }
    }
    if constexpr (kOut) {
        __syncthreads();
        write_out(blocks - 1);
    }
}

// A few tokens [begin, end) straight from global memory.
template <int N, bool kGate>
__device__ __forceinline__ void sel_few(const SelParams &p, SelLane &me, int begin, int end, int ch, bool valid,
                                        float D, float bias)
{
    constexpr int kChannels = 32 / (N / kStates);
    const int part = (threadIdx.x & 31) / kChannels;
    for (int64_t t = begin; t < end; ++t) {
        const float x = __bfloat162float(p.x[t * p.x_stride + ch]);
        const float v = __bfloat162float(p.dt[t * p.dt_stride + ch]) + bias;
        const float z = kGate ? __bfloat162float(p.z[t * p.z_stride + ch]) : 0.f;
        const float dt = p.softplus ? step_of(v) : v;
        float sum = me.token(dt, dt * x, p.B + t * p.b_stride + part * kStates,
                             p.C + t * p.c_stride + part * kStates);
#pragma unroll
        for (int o = kChannels; o < 32; o <<= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
        float y = fmaf(D, x, sum);
        if constexpr (kGate)
            y *= silu_f32(z);
        if (part == 0 && valid)
            p.y[t * p.y_stride + ch] = __float2bfloat16_rn(y);
    }
}

// A tile of channels as one of its lanes sees it.
template <int N>
struct SelPlace {
    int col0, ch, part;
    bool valid;                               // (lanes past the last channel follow one that is there)
    int64_t at;                               // the lane's states in a slot
    int64_t states;                           // those of a slot

    __device__ __forceinline__ SelPlace(const SelParams &p, int tile)
    {
        constexpr int kChannels = SelShared<N, 16>::kChannels;
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        part = lane / kChannels;
        col0 = tile * SelShared<N, 16>::kCols;
        ch = col0 + warp * kChannels + lane % kChannels;
        valid = ch < p.channels;
        ch = valid ? ch : 0;
        states = static_cast<uint32_t>(p.channels) * N;
        at = static_cast<int64_t>(ch) * N + part * kStates;
    }
};

// A whole sequence, or the first chunk of a cut one: from the slot's states; these go to the slot,
// or to the chunk's end.
template <int N, bool kGate>
__device__ __forceinline__ void sel_first(const SelParams &p, const SelPlace<N> &me_at, SelShared<N, 16> &s,
                                          const SelUnit &u)
{
    SelLane me;
    me.load_decays(p.A + me_at.at);
    const float D = p.D ? p.D[me_at.ch] : 0.f, bias = p.dt_bias ? p.dt_bias[me_at.ch] : 0.f;
    const int64_t slot = seq_slot(p.s, u.seq);
#pragma unroll
    for (int n = 0; n < kStates; ++n)
        me.h[n] = 0.f;
    if (slot >= 0 && p.s.has_init && p.s.has_init[u.seq])
        load_states(p.pool, p.pool_bf16, slot * me_at.states + me_at.at, me.h);
    float total = 0.f;
    if (u.end - u.begin > kFew)
        sel_tokens<N, kGate, true>(p, s, me, u.begin, u.end, me_at.col0, D, bias, total);
    else
        sel_few<N, kGate>(p, me, u.begin, u.end, me_at.ch, me_at.valid, D, bias);
    if (!me_at.valid)
        return;
    if (u.cut)
        store_states(p.ends, false, u.ends * me_at.states + me_at.at, me.h);
    else if (slot >= 0)
        store_states(p.pool, p.pool_bf16, slot * me_at.states + me_at.at, me.h);
}

// The tokens of a whole sequence, or of a chunk that is not its sequence's first.  (With the CTAs
// of an SM asked for: without, ptxas keeps to 80 registers and orders the code for that, 560 us
// for two prompts of 9,763 tokens in all instead of 430, with blocks of 16 tokens.  Three asked
// for and not the four that there are from 16 states on, which it orders worse; with 8 there are two.)
template <int N, bool kGate, int kBlock>
__global__ void __launch_bounds__(kScanThreads, kBlock == 32 ? 2 : 3) selective_scan_kernel(const __grid_constant__ SelParams p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    const SelPlace<N> me_at(p, blockIdx.x % p.tiles);
    const int unit = blockIdx.x / p.tiles;
    pdl_wait();
    SelUnit u = {unit, 0, 0, 0, 0, 0, 1, 0};
    if (p.units) {
        if (unit >= (p.behind ? p.header->ends : p.header->units))
            return;
        u = p.units[unit];
    } else if (!seq_rows(p.s.qsl, p.s.total_len, p.s.errors, unit, u.begin, u.end) || u.end - u.begin <= p.few) {
        return;
    }
    SelLane me;
    me.load_decays(p.A + me_at.at);
    const float D = p.D ? p.D[me_at.ch] : 0.f, bias = p.dt_bias ? p.dt_bias[me_at.ch] : 0.f;
    const int64_t slot = seq_slot(p.s, u.seq);
#pragma unroll
    for (int n = 0; n < kStates; ++n)
        me.h[n] = 0.f;
    if (u.k > 0) {
#pragma unroll 4
        for (int64_t e = u.ends; e < u.ends + u.k; ++e) {
            float own[kStates];
            load_states(p.ends, false, e * me_at.states + me_at.at, own);
            const float sum = p.sums[e * p.channels + me_at.ch];
#pragma unroll
            for (int n = 0; n < kStates; ++n)
                me.h[n] = e == u.ends ? own[n] : fmaf(ptx::ex2(sum * me.decay(n)), me.h[n], own[n]);
        }
    } else if (slot >= 0 && p.s.has_init && p.s.has_init[u.seq]) {
        load_states(p.pool, p.pool_bf16, slot * me_at.states + me_at.at, me.h);
    }
    float total = 0.f;
    if (u.end - u.begin > kFew)
        sel_tokens<N, kGate, true>(p, *reinterpret_cast<SelShared<N, kBlock> *>(smem), me, u.begin, u.end, me_at.col0, D,
                                   bias, total);
    else
        sel_few<N, kGate>(p, me, u.begin, u.end, me_at.ch, me_at.valid, D, bias);
    if (u.last && slot >= 0 && me_at.valid)
        store_states(p.pool, p.pool_bf16, slot * me_at.states + me_at.at, me.h);
}

// Whole sequences and chunks: first ones, and of those between the first and the last the states
// from zero and the steps' sum alone.
template <int N, bool kGate>
__global__ void __launch_bounds__(kScanThreads, kResident) selective_first_kernel(const __grid_constant__ SelParams p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    auto &shared = *reinterpret_cast<SelShared<N, 16> *>(smem);
    const SelPlace<N> me_at(p, blockIdx.x % p.tiles);
    const int unit = blockIdx.x / p.tiles;
    pdl_wait();
    if (unit >= p.header->units)
        return;
    const SelUnit u = p.units[unit];
    if (u.k == 0) {
        sel_first<N, kGate>(p, me_at, shared, u);
        return;
    }
    SelLane me;
    me.load_decays(p.A + me_at.at);
#pragma unroll
    for (int n = 0; n < kStates; ++n)
        me.h[n] = 0.f;
    float total = 0.f;
    sel_tokens<N, false, false>(p, shared, me, u.begin, u.end, me_at.col0, 0.f, p.dt_bias ? p.dt_bias[me_at.ch] : 0.f,
                                total);
    if (!me_at.valid)
        return;
    const int64_t end = u.ends + u.k;
    store_states(p.ends, false, end * me_at.states + me_at.at, me.h);
    if (me_at.part == 0)
        p.sums[end * p.channels + me_at.ch] = total;
}

// Sequences of at most p.few tokens, single ones as a rule.  A CTA takes every `groups`-th
// sequence for its tile of channels and looks kScanThreads of them up at once; its warps
// are on their own otherwise, each with the states and first tokens of kAhead sequences in
// registers, on their way while it works on one.
constexpr int kStepResident = 6;      // CTAs of an SM
constexpr int kAhead = 2;             // sequences that a warp holds

struct alignas(16) SelSequence {
    uint32_t slot;                    // or SSD_NO_SLOT
    int32_t begin, tokens;            // (tokens < 0: not this kernel's, or its offsets are none)
    int32_t has;                      // an initial state
};

template <int N, bool kGate, bool kBf16>
__global__ void __launch_bounds__(kScanThreads, kStepResident) selective_step_kernel(const __grid_constant__ SelParams p)
{
    // Neighbouring lanes are a channel's, and a load of theirs takes what lies side by side: 16
    // bytes of states each, four fp32 or eight bf16.
    constexpr int kLanes = N / kStates;
    constexpr int kLoads = kBf16 ? 1 : 2;     // of 16 bytes, of a lane's states
    __shared__ SelSequence s_seq[kScanThreads];
    const int part = threadIdx.x % kLanes;
    const int there = static_cast<int>(blockIdx.x % p.tiles) * SelShared<N, 16>::kCols + threadIdx.x / kLanes;
    const bool valid = there < p.channels;    // (lanes past the last channel follow one that is there)
    const int ch = valid ? there : 0;
    const int64_t states = static_cast<int64_t>(p.channels) * N;
    // the first state of the lane's four with index i
    auto four = [&](int i) { return kBf16 ? part * kStates + 4 * i : (i * kLanes + part) * 4; };
    const int groups = gridDim.x / p.tiles, tid = threadIdx.x;
    pdl_wait();
    struct Token {
        uint2 B[2], C[2];
        __nv_bfloat16 x, dt, z;
    };
    const __nv_bfloat16 none = __float2bfloat16_rn(0.f);
    auto load_token = [&](int64_t t) {
        Token v;
        v.x = p.x[t * p.x_stride + ch];
        v.dt = p.dt[t * p.dt_stride + ch];
        v.z = kGate ? p.z[t * p.z_stride + ch] : none;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v.B[i] = *reinterpret_cast<const uint2 *>(p.B + t * p.b_stride + four(i));
            v.C[i] = *reinterpret_cast<const uint2 *>(p.C + t * p.c_stride + four(i));
        }
        return v;
    };
    using Element = std::conditional_t<kBf16, __nv_bfloat16, float>;
    Element *pool = static_cast<Element *>(p.pool) + static_cast<int64_t>(ch) * N;
    struct Item {
        SelSequence q;
        uint4 state[kLoads];
        Token token;
    };
    auto load = [&](Item &it, int i, int count) {
        it.q = i < count ? s_seq[i] : SelSequence{SSD_NO_SLOT, 0, -1, 0};
#pragma unroll
        for (int k = 0; k < kLoads; ++k)
            it.state[k] = it.q.has ? *reinterpret_cast<const uint4 *>(pool + it.q.slot * states + four(k))
                                   : make_uint4(0, 0, 0, 0);
        if (it.q.tokens > 0)
            it.token = load_token(it.q.begin);
    };
    uint64_t a[kStates / 2];                  // A log2(e), two states each
#pragma unroll
    for (int k = 0; k < kStates / 4; ++k) {
        const float4 v = __ldg(reinterpret_cast<const float4 *>(p.A + static_cast<int64_t>(ch) * N + four(k)));
        a[2 * k] = ptx::pack2(v.x * kLog2e, v.y * kLog2e);
        a[2 * k + 1] = ptx::pack2(v.z * kLog2e, v.w * kLog2e);
    }
    const float D = p.D ? p.D[ch] : 0.f, bias = p.dt_bias ? p.dt_bias[ch] : 0.f;
    uint64_t h[kStates / 2];
    auto step = [&](const Token &v, int64_t t) {
        const float x = __bfloat162float(v.x), raw = __bfloat162float(v.dt) + bias;
        const float dt = p.softplus ? step_of(raw) : raw, u = dt * x;
        const uint64_t dt2 = ptx::pack2(dt, dt), u2 = ptx::pack2(u, u);
        const uint32_t B[4] = {v.B[0].x, v.B[0].y, v.B[1].x, v.B[1].y};
        const uint32_t C[4] = {v.C[0].x, v.C[0].y, v.C[1].x, v.C[1].y};
        uint64_t sum2 = 0;
#pragma unroll
        for (int k = 0; k < kStates / 2; ++k) {
            float e0, e1;
            ptx::unpack2(ptx::mul2(dt2, a[k]), e0, e1);
            const uint64_t b = ptx::pack2(__uint_as_float(B[k] << 16), __uint_as_float(B[k] & 0xffff0000u));
            const uint64_t c = ptx::pack2(__uint_as_float(C[k] << 16), __uint_as_float(C[k] & 0xffff0000u));
            h[k] = ptx::fma2(ptx::pack2(ptx::ex2(e0), ptx::ex2(e1)), h[k], ptx::mul2(u2, b));
            sum2 = ptx::fma2(h[k], c, sum2);
        }
        float sum, other;
        ptx::unpack2(sum2, sum, other);
        sum += other;
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
        float y = fmaf(D, x, sum);
        if constexpr (kGate)
            y *= silu_f32(__bfloat162float(v.z));
        if (part == 0 && valid)
            p.y[t * p.y_stride + ch] = __float2bfloat16_rn(y);
    };
    auto work = [&](const Item &it) {
        if (it.q.tokens < 0)
            return;
        if constexpr (kBf16) {
            const uint32_t w[4] = {it.state[0].x, it.state[0].y, it.state[0].z, it.state[0].w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                h[k] = ptx::pack2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
        } else {
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                h[2 * k] = ptx::pack2(__uint_as_float(it.state[k].x), __uint_as_float(it.state[k].y));
                h[2 * k + 1] = ptx::pack2(__uint_as_float(it.state[k].z), __uint_as_float(it.state[k].w));
            }
        }
        if (it.q.tokens > 0) {
            step(it.token, it.q.begin);
            // (loading a further token ahead would cost registers that the others need: 96
            // single tokens 28 us instead of 22)
            for (int i = 1; i < it.q.tokens; ++i)
                step(load_token(it.q.begin + i), it.q.begin + i);
        }
        if (it.q.slot == SSD_NO_SLOT || !valid)
            return;
        float v[kStates];
#pragma unroll
        for (int k = 0; k < kStates / 2; ++k)
            ptx::unpack2(h[k], v[2 * k], v[2 * k + 1]);
        Element *to = pool + it.q.slot * states;
        if constexpr (kBf16) {
            *reinterpret_cast<uint4 *>(to + four(0)) = round8(v);
        } else {
            *reinterpret_cast<float4 *>(to + four(0)) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4 *>(to + four(1)) = make_float4(v[4], v[5], v[6], v[7]);
        }
    };
    for (int b0 = blockIdx.x / p.tiles; b0 < p.s.batch; b0 += kScanThreads * groups) {
        __syncthreads();      // everybody is done with the sequences before
        const int count = min(kScanThreads, (p.s.batch - b0 + groups - 1) / groups);
        if (tid < count) {
            const int b = b0 + tid * groups;
            int32_t begin, end;
            SelSequence q = {SSD_NO_SLOT, 0, -1, 0};
            if (seq_rows(p.s.qsl, p.s.total_len, p.s.errors, b, begin, end)) {
                q.slot = static_cast<uint32_t>(seq_slot(p.s, b));
                q.begin = begin;
                q.tokens = end - begin <= p.few ? end - begin : -1;
                q.has = q.tokens >= 0 && q.slot != SSD_NO_SLOT && p.s.has_init && p.s.has_init[b];
            }
            s_seq[tid] = q;
        }
        __syncthreads();
        Item item[kAhead];
#pragma unroll
        for (int k = 0; k + 1 < kAhead; ++k)
            load(item[k], k, count);
        for (int i = 0; i < count; i += kAhead)
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                load(item[(k + kAhead - 1) % kAhead], i + k + kAhead - 1, count);
                work(item[k]);
            }
    }
}

// Ends of chunks of a call, at most: a cut sequence's chunks are no shorter than sel_chunk,
// and its last has no end.
int64_t sel_ends(int64_t total_len, int32_t chunk) { return total_len / chunk; }

struct SelLayout {
    size_t units, later, ends, sums, total;
};
SelLayout sel_layout(int64_t total_len, int32_t batch, int32_t channels, int32_t dstate, int64_t ends)
{
    SelLayout L;
    size_t off = (sizeof(SelHeader) + 255) & ~size_t{255};
    auto take = [&](int64_t bytes) {
        const size_t at = off;
        off = (off + static_cast<size_t>(bytes) + 255) & ~size_t{255};
        return at;
    };
    const int64_t states = static_cast<int64_t>(channels) * dstate * 4;
    L.units = take((ends + batch) * static_cast<int64_t>(sizeof(SelUnit)));
    L.later = take(ends * static_cast<int64_t>(sizeof(SelUnit)));
    L.ends = take(ends * states);
    L.sums = take(ends * channels * 4);
    L.total = off;
    return L;
}

// Bytes for these sizes and all that are not larger: sel_chunk gives at most kFullWarps /
// warps ends, with channels dstate / 256 warps at least, and none below kMinChunk.
size_t sel_bytes(int64_t total_len, int32_t batch, int32_t channels, int32_t dstate)
{
    const int64_t states = static_cast<int64_t>(channels) * dstate, ends = total_len / kMinChunk;
    const int64_t held = std::min<int64_t>(ends * states, int64_t{kFullWarps} * 32 * kStates);
    return static_cast<size_t>(held * 4 + held / kStates * 4 +
                               (2 * std::min<int64_t>(ends, kFullWarps) + batch) * static_cast<int64_t>(sizeof(SelUnit)) +
                               6 * 256 + sizeof(SelHeader));
}

template <int N, bool kGate>
cudaError_t launch(SelParams &p, cudaStream_t stream)
{
    constexpr int kCols = SelShared<N, 16>::kCols, kBytes = sizeof(SelShared<N, 16>);
    p.tiles = (p.channels + kCols - 1) / kCols;
    int device = 0, sms = 0;
    if (cudaGetDevice(&device) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
        return cudaErrorInvalidDevice;
    // Where most sequences have few tokens, those have a kernel of their own, without shared
    // memory or a list (96 of two tokens, 8,192 channels: 35.5 us with both kernels, 63 in the other
    // one alone; 24 sequences of 72 tokens on average, twenty of them of one: 69.5 and 65.9).  It
    // takes all of them, whatever their lengths, when there are as many tokens as sequences, a step
    // of single tokens (96 of them 22 us, 25 with both kernels).  Fewer tokens than sequences are a
    // batch with empty ones, whose others may be long: one of 256 and 255 single tokens among 256
    // empty ones, 2,048 channels, 199 us there and 46 with both.  No more CTAs than are resident at
    // once.
    const bool alone = p.s.total_len == p.s.batch || p.s.total_len <= kFew;
    p.few = alone                                        ? INT32_MAX
            : p.s.total_len <= int64_t{kFew} * p.s.batch ? kFew
                                                         : -1;
    if (p.few >= 0) {
        const int64_t groups = std::min<int64_t>(p.s.batch, std::max(1, kStepResident * sms / p.tiles));
        const cudaError_t e =
            launch_pdl(p.pool_bf16 ? selective_step_kernel<N, kGate, true> : selective_step_kernel<N, kGate, false>,
                       dim3(static_cast<unsigned>(p.tiles * groups)), kScanThreads, stream, p);
        if (e != cudaSuccess || alone)
            return e;
    }
    // Calls of few tokens are not cut, and neither are those whose sequences have warps for two
    // thirds of the schedulers each: whole, without the list, the idle CTAs and in blocks of 32 tokens,
    // they take less as a rule (one of 500 and one of 9,763 tokens, 8,192 channels: 40 and 532 us
    // cut, 30.5 and 505 whole; of 16,384 channels, which the list leaves whole: 71 and 1,206, without it
    // 47 and 806; two prompts of 9,763 tokens in all, 8,192 channels: 473 and 430 then; but one of
    // 9,763, 6,528 channels: 457 and 503).
    const bool may_cut = p.s.total_len >= 2 * int64_t{p.chunk} && 3 * p.warps < 8 * sms;
    const int64_t ends = may_cut ? sel_ends(p.s.total_len, p.chunk) : 0;
    if (!may_cut)
        p.chunk = 0;
    // (those of more than few tokens are not many; the list leaves the others out)
    const int64_t most = p.few < 0 ? p.s.batch : std::min<int64_t>(p.s.batch, p.s.total_len / (p.few + 1));
    int64_t whole = static_cast<int64_t>(p.tiles) * p.s.batch;
    const bool listed = ends || whole > int64_t{sel_resident<N, 16>(kResident)} * sms;
    if (listed)
        whole = p.tiles * most;
    static SmemOptIn s_scan, s_long, s_first;
    auto go = [&](auto kernel, SmemOptIn &opted, int64_t ctas, int bytes) {
        const cudaError_t e = ensure_max_smem(reinterpret_cast<const void *>(kernel), opted);
        return e != cudaSuccess ? e
                                : launch_pdl_smem(kernel, dim3(static_cast<unsigned>(ctas)), kScanThreads, bytes, stream, p);
    };
    if (listed) {
        cudaError_t e = launch_pdl(selective_plan_kernel, dim3(1), kPlanThreads, stream, p);
        if (e == cudaSuccess)
            e = ends ? go(selective_first_kernel<N, kGate>, s_first, p.tiles * ends + whole, kBytes)
                     : go(selective_scan_kernel<N, kGate, 16>, s_scan, whole, kBytes);
        if (e == cudaSuccess && ends) {
            p.units = p.later;
            p.behind = 1;
            e = go(selective_scan_kernel<N, kGate, 16>, s_scan, p.tiles * ends, kBytes);
        }
        return e;
    }
    // At most two CTAs an SM (one with 8 states, whose blocks of 32 leave no room for two): blocks of
    // 32 tokens, fewer barriers for more shared memory (two prompts of 9,763 tokens in all, 8,192
    // channels: 429 us with 16, 399 with 32; with four CTAs an SM, 8 of 1,000 tokens and 5,120
    // channels: 214 and 227; two of 2,000 tokens, 16,384 channels of 8 states, 256 CTAs: 220 and 276).
    p.units = nullptr;
    return whole <= sel_resident<N, 32>(2) * sms
               ? go(selective_scan_kernel<N, kGate, 32>, s_long, whole, sizeof(SelShared<N, 32>))
               : go(selective_scan_kernel<N, kGate, 16>, s_scan, whole, kBytes);
}

template <int N>
cudaError_t launch(SelParams &p, cudaStream_t stream)
{
    return p.z ? launch<N, true>(p, stream) : launch<N, false>(p, stream);
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
    if (!ssd::sel_sizes(total_len, batch, channels, dstate))
        return 0;
    return ssd::sel_bytes(total_len, batch, channels, dstate);
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
    if (std::max({t.y, t.x, t.dt, t.z, t.B, t.C}) > INT32_MAX)
        return SSD_ERR_UNSUPPORTED;
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
    p.y_stride = static_cast<int32_t>(t.y);
    p.x_stride = static_cast<int32_t>(t.x);
    p.dt_stride = static_cast<int32_t>(t.dt);
    p.b_stride = static_cast<int32_t>(t.B);
    p.c_stride = static_cast<int32_t>(t.C);
    p.z_stride = static_cast<int32_t>(t.z);
    p.channels = channels;
    p.softplus = dt_softplus != 0;
    p.pool_bf16 = pool_type == SSD_POOL_BF16;
    p.chunk = sel_chunk(total_len, channels, dstate);
    p.warps = static_cast<int32_t>(sel_warps(channels, dstate));
    const SelLayout L = sel_layout(total_len, batch, channels, dstate, sel_ends(total_len, p.chunk));
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.header = reinterpret_cast<SelHeader *>(ws);
    p.units = reinterpret_cast<SelUnit *>(ws + L.units);
    p.later = reinterpret_cast<SelUnit *>(ws + L.later);
    p.ends = reinterpret_cast<float *>(ws + L.ends);
    p.sums = reinterpret_cast<float *>(ws + L.sums);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = dstate == 8    ? launch<8>(p, s)
                          : dstate == 16 ? launch<16>(p, s)
                          : dstate == 32 ? launch<32>(p, s)
                                         : launch<64>(p, s);
    return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
