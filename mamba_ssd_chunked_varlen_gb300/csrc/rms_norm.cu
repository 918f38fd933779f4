// Root-mean-square norm over groups of columns, with a residual's addition or a gate
// before it and an output in bf16 or in 8-bit codes:
//
//     s = x, x + residual (written back) or x silu(gate)
//     y = s w / sqrt(mean s^2 + eps);   codes: a = max|y|, code = round(y M / a), scale = a / M
//
// A segment is one row's group.  It is read once and stays in registers, eight values
// a load, between the sum of squares, the largest magnitude and the output: memory
// bounds it with a residual or to bf16.  Segments of up to 1,024 columns are a warp's or less
// (eight lanes up to 64, sixteen up to 128), longer ones a CTA's.  There, for codes, y is (s w) r with
// r = 1 / sqrt(...): a product with r > 0 keeps the order of magnitudes through its rounding, so
// that max|y| is max|s w| r, and one barrier serves the sum and the largest (4,093 rows of
// 5,120 to int8: 29.1 us with two, 27.1 with one, 25.8 with rows in turn; a warp's weights
// would be registers that it needs, 8,191 rows of 8 gated groups to int8: 73 us with them, 68
// without).  With a residual, 4,093 rows of 5,120 to bf16 take 26.9 us, 92 % of the measured copy
// rate, to int8 25.8, 84 %; 8,191 rows of 8 gated groups to bf16 65, 90 %.
//
// Instructions bound codes without a residual (8,191 rows of 8,192 to int8: plain 47 us, 63 % of
// the copy rate, gated 86, 57 %), and the 64 registers of a CTA of 1,024 threads those of more
// than 16,384 columns, whose 32 values and 32 weights a thread do not fit: 360 to 400 bytes a thread
// go to local memory and back (2,047 rows of 32,768 to int8: plain 89 us, 33 %, with a residual 132,
// 52 %; to bf16, where the weights are loaded late and nothing spills, 60 and 87 us).  Rows in turn spill
// 52 bytes to codes with a gate, 44 with a residual, 16 to bf16 with a gate.
#include <algorithm>

#include "layer_common.cuh"

namespace ssd {
namespace {

constexpr int kNormThreads = 128;    // threads of a CTA that takes several segments
constexpr int kNormMaxVecs = 4;      // loads of eight values that a thread holds

enum NormInput { kPlain, kResidual, kGate };

struct NormParams {
    void *y;
    float *scale;
    const __nv_bfloat16 *x, *gate;
    __nv_bfloat16 *residual;
    const float *weight;
    int64_t rows, segments, y_stride, x_stride, residual_stride, gate_stride;
    int32_t groups, cols;            // columns of a group
    float eps;
};

// Sum of v and largest of m over a segment's kLanes lanes, or (0) all of the CTA's.
template <int kLanes, bool kTop>
__device__ __forceinline__ void reduce(float &v, uint32_t &m, float2 *scratch)
{
    constexpr int kWidth = kLanes ? kLanes : 32;
#pragma unroll
    for (int o = kWidth / 2; o > 0; o >>= 1) {
        v += __shfl_xor_sync(0xffffffffu, v, o);
        if constexpr (kTop)
            m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    if constexpr (kLanes == 0) {
        const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        if (lane == 0)
            scratch[threadIdx.x >> 5] = make_float2(v, __uint_as_float(m));
        __syncthreads();
        const float2 part = lane < warps ? scratch[lane] : make_float2(0.f, 0.f);
        v = part.x;
        m = __float_as_uint(part.y);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            v += __shfl_xor_sync(0xffffffffu, v, o);
        if constexpr (kTop)
            m = __reduce_max_sync(0xffffffffu, m);
    }
}

// Whether a CTA takes row after row of its group, whose weights it keeps, with the next row's
// loads ahead.  (8,191 rows of 8,192 columns, a row a CTA against rows in turn: plain to int8 65
// and 47 us, gated to bf16 65 and 61, to int8 89 and 85, with a residual to int8 80 and 76; but to
// bf16 with a residual 78 and 88, as three CTAs of 40 registers a thread load more than two of 64.)
constexpr bool norm_in_turn(int type, int in) { return type != SSD_KV_BF16 || in != kResidual; }

// kLanes: lanes of a segment, 0 for a CTA; kThreads: threads of a CTA at most; kResident: CTAs of
// so many threads that an SM's registers are to suffice for.
template <int kType, int kIn, int kVecs, int kLanes, int kThreads, int kResident>
__global__ void __launch_bounds__(kThreads, kResident)
norm_kernel(const __grid_constant__ NormParams p)
{
    constexpr bool kCodes = kType != SSD_KV_BF16, kEarly = kCodes && kLanes == 0;
    __shared__ float2 s_part[2][32];
    const int tid = kLanes ? threadIdx.x % (kLanes ? kLanes : 1) : threadIdx.x;
    const int step = (kLanes ? kLanes : blockDim.x) * 8;
    const int64_t seg = kLanes ? static_cast<int64_t>(blockIdx.x) * (kThreads / (kLanes ? kLanes : 1)) +
                                     threadIdx.x / (kLanes ? kLanes : 1)
                               : blockIdx.x;
    pdl_wait();
    // (lanes without a segment go along: the others' shuffles name them)
    const bool there = seg < p.segments;
    const int64_t row = there ? seg / p.groups : 0;
    const int col0 = there ? static_cast<int>(seg % p.groups) * p.cols : 0;
    const int cols = there ? p.cols : 0;
    float s[kVecs][8], w[kVecs][8];
    uint4 raw[kVecs], other[kVecs];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        const int c = v * step + tid * 8;
        raw[v] = other[v] = make_uint4(0, 0, 0, 0);
        if (c < cols) {
            raw[v] = *reinterpret_cast<const uint4 *>(p.x + row * p.x_stride + col0 + c);
            if constexpr (kIn == kResidual)
                other[v] = *reinterpret_cast<const uint4 *>(p.residual + row * p.residual_stride + col0 + c);
            if constexpr (kIn == kGate)
                other[v] = *reinterpret_cast<const uint4 *>(p.gate + row * p.gate_stride + col0 + c);
        }
    }
    auto weights = [&](int v) {
        const int c = v * step + tid * 8;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 f = p.weight && c < cols
                                 ? __ldg(reinterpret_cast<const float4 *>(p.weight + col0 + c) + i)
                                 : make_float4(1.f, 1.f, 1.f, 1.f);
            w[v][4 * i] = f.x;
            w[v][4 * i + 1] = f.y;
            w[v][4 * i + 2] = f.z;
            w[v][4 * i + 3] = f.w;
        }
    };
    if constexpr (kEarly)
#pragma unroll
        for (int v = 0; v < kVecs; ++v)
            weights(v);
    float sum = 0.f;
    uint32_t top = 0;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        widen8(raw[v], s[v]);
        if constexpr (kIn != kPlain) {
            float o[8];
            widen8(other[v], o);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                s[v][k] = kIn == kResidual ? s[v][k] + o[k] : s[v][k] * silu_f32(o[k]);
        }
        if constexpr (kIn == kResidual) {
            const int c = v * step + tid * 8;
            if (c < cols)
                *reinterpret_cast<uint4 *>(p.residual + row * p.residual_stride + col0 + c) = round8(s[v]);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            sum = fmaf(s[v][k], s[v][k], sum);
            if constexpr (kEarly)
                top = max(top, __float_as_uint(s[v][k] * w[v][k]) & 0x7fffffffu);
        }
    }
    reduce<kLanes, kEarly>(sum, top, s_part[0]);
    float r = rsqrtf(sum / static_cast<float>(p.cols) + p.eps);
    // (all of a segment's threads take this way or none; in a warp of several segments
    // all lanes do when one segment has to)
    const bool again = !(sum < __int_as_float(0x7f800000));
    if (kLanes ? __any_sync(0xffffffffu, again) : again) {
        // squares out of range (or infinities and NaN): once more on s 2^-80, where eps is
        // nothing beside the mean
        const float by = again ? 0x1p-80f : 1.f;
        sum = 0.f;
        top = 0;
#pragma unroll
        for (int v = 0; v < kVecs; ++v)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                s[v][k] *= by;
                sum = fmaf(s[v][k], s[v][k], sum);
                if constexpr (kEarly)
                    top = max(top, __float_as_uint(s[v][k] * w[v][k]) & 0x7fffffffu);
            }
        reduce<kLanes, kEarly>(sum, top, s_part[1]);
        if (again)
            r = rsqrtf(sum / static_cast<float>(p.cols));
    }
    if constexpr (!kCodes) {
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            const int c = v * step + tid * 8;
            weights(v);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                s[v][k] = s[v][k] * r * w[v][k];
            if (c < cols)
                *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.y) + row * p.y_stride + col0 + c) =
                    round8(s[v]);
        }
    } else {
        constexpr float kTop = kType == SSD_KV_INT8 ? kInt8Max : kE4m3Max;
        if constexpr (!kEarly) {
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
                weights(v);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    s[v][k] = s[v][k] * r * w[v][k];
                    top = max(top, v * step + tid * 8 < cols ? __float_as_uint(s[v][k]) & 0x7fffffffu : 0u);
                }
            }
            float none = 0.f;
            reduce<kLanes, true>(none, top, s_part[0]);
        }
        const float largest = kEarly ? __uint_as_float(top) * r : __uint_as_float(top);
        const bool bad = !(largest < __int_as_float(0x7f800000));
        const float a = fmaxf(largest, kKvTiny), inv = __fdiv_rn(kTop, a);
        if (there && tid == 0)
            p.scale[seg] = bad ? __int_as_float(0x7fffffff) : __fdiv_rn(a, kTop);
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            const int c = v * step + tid * 8;
            if constexpr (kEarly)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    s[v][k] = s[v][k] * w[v][k] * r;
            if (c < cols)
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.y) + row * p.y_stride + col0 + c) =
                    bad ? make_uint2(0, 0) : encode8<kType>(s[v], inv);
        }
    }
}

// The same for a group's rows one after the other: blockIdx.x % groups is the CTA's group.  (One
// barrier a row: its scratch is another one than the row's before.)
template <int kType, int kIn, int kThreads, int kResident>
__global__ void __launch_bounds__(kThreads, kResident) norm_rows_kernel(const __grid_constant__ NormParams p)
{
    constexpr bool kCodes = kType != SSD_KV_BF16;
    constexpr int kVecs = 2;
    __shared__ float2 s_part[3][32];
    const int step = blockDim.x * 8, group = static_cast<int>(blockIdx.x % p.groups), row_step = gridDim.x / p.groups;
    const int col0 = group * p.cols;
    pdl_wait();
    float s[kVecs][8], w[kVecs][8];
    uint4 raw[kVecs], other[kVecs];
    const int at0 = col0 + threadIdx.x * 8;
    auto load = [&](int64_t row) {
        const __nv_bfloat16 *x = p.x + row * p.x_stride + at0;
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            const int c = v * step + threadIdx.x * 8;
            raw[v] = other[v] = make_uint4(0, 0, 0, 0);
            if (c < p.cols && row < p.rows) {
                raw[v] = *reinterpret_cast<const uint4 *>(x + v * step);
                if constexpr (kIn == kResidual)
                    other[v] = *reinterpret_cast<const uint4 *>(p.residual + row * p.residual_stride + col0 + c);
                if constexpr (kIn == kGate)
                    other[v] = *reinterpret_cast<const uint4 *>(p.gate + row * p.gate_stride + col0 + c);
            }
        }
    };
    int64_t row = blockIdx.x / p.groups;
    load(row);
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        const int c = v * step + threadIdx.x * 8;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 f = p.weight && c < p.cols
                                 ? __ldg(reinterpret_cast<const float4 *>(p.weight + col0 + c) + i)
                                 : make_float4(1.f, 1.f, 1.f, 1.f);
            w[v][4 * i] = f.x;
            w[v][4 * i + 1] = f.y;
            w[v][4 * i + 2] = f.z;
            w[v][4 * i + 3] = f.w;
        }
    }
    for (int turn = 0; row < p.rows; row += row_step, turn ^= 1) {
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            widen8(raw[v], s[v]);
            if constexpr (kIn != kPlain) {
                float o[8];
                widen8(other[v], o);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    s[v][k] = kIn == kResidual ? s[v][k] + o[k] : s[v][k] * silu_f32(o[k]);
            }
        }
        load(row + row_step);
        float sum = 0.f;
        uint32_t top = 0;
        auto add = [&](int v) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                sum = fmaf(s[v][k], s[v][k], sum);
                if constexpr (kCodes)
                    top = max(top, __float_as_uint(s[v][k] * w[v][k]) & 0x7fffffffu);
            }
        };
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            const int c = v * step + threadIdx.x * 8;
            if (kIn == kResidual && c < p.cols)
                *reinterpret_cast<uint4 *>(p.residual + row * p.residual_stride + col0 + c) = round8(s[v]);
            add(v);
        }
        reduce<0, kCodes>(sum, top, s_part[turn]);
        float r = rsqrtf(sum / static_cast<float>(p.cols) + p.eps);
        if (!(sum < __int_as_float(0x7f800000))) {     // (the same in all threads; as above)
            sum = 0.f;
            top = 0;
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    s[v][k] *= 0x1p-80f;
                add(v);
            }
            reduce<0, kCodes>(sum, top, s_part[2]);
            r = rsqrtf(sum / static_cast<float>(p.cols));
        }
        float inv = 0.f;
        bool bad = false;
        if constexpr (kCodes) {
            constexpr float kTop = kType == SSD_KV_INT8 ? kInt8Max : kE4m3Max;
            const float largest = __uint_as_float(top) * r, a = fmaxf(largest, kKvTiny);
            bad = !(largest < __int_as_float(0x7f800000));
            inv = __fdiv_rn(kTop, a);
            if (threadIdx.x == 0)
                p.scale[row * p.groups + group] = bad ? __int_as_float(0x7fffffff) : __fdiv_rn(a, kTop);
        }
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            const int c = v * step + threadIdx.x * 8;
            const int64_t at = row * p.y_stride + col0 + c;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                s[v][k] = kCodes ? s[v][k] * w[v][k] * r : s[v][k] * r * w[v][k];
            if (c < p.cols) {
                if constexpr (kCodes)
                    *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.y) + at) =
                        bad ? make_uint2(0, 0) : encode8<kType>(s[v], inv);
                else
                    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.y) + at) = round8(s[v]);
            }
        }
    }
}

template <int kType, int kIn>
cudaError_t launch(const NormParams &p, cudaStream_t stream)
{
    const int loads = p.cols / 8;
    // up to a warp a segment while its lanes hold four loads at most: no barrier
    if (loads <= 4 * 32) {
        auto go = [&](auto kernel, int lanes) {
            const int64_t each = kNormThreads / lanes;
            return launch_pdl(kernel, dim3(static_cast<unsigned>((p.segments + each - 1) / each)), kNormThreads, stream,
                              p);
        };
        return loads <= 8    ? go(norm_kernel<kType, kIn, 1, 8, kNormThreads, 8>, 8)
               : loads <= 16 ? go(norm_kernel<kType, kIn, 1, 16, kNormThreads, 8>, 16)
               : loads <= 32 ? go(norm_kernel<kType, kIn, 1, 32, kNormThreads, 8>, 32)
               : loads <= 64 ? go(norm_kernel<kType, kIn, 2, 32, kNormThreads, 8>, 32)
                             : go(norm_kernel<kType, kIn, 4, 32, kNormThreads, 8>, 32);
    }
    constexpr bool kInTurn = norm_in_turn(kType, kIn);
    const int vecs = loads <= 2 * (kInTurn ? 1024 : 512) ? 2 : kNormMaxVecs;
    const int threads = (loads + 32 * vecs - 1) / (32 * vecs) * 32;
    if constexpr (kInTurn)
        if (vecs == 2) {
            // as many CTAs as 64 registers a thread leave room for, each with rows of one group
            int device = 0, sms = 0;
            if (cudaGetDevice(&device) != cudaSuccess ||
                cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
                return cudaErrorInvalidDevice;
            const int64_t resident = static_cast<int64_t>(1024 / threads) * sms;
            const int64_t each = std::min(std::max<int64_t>(1, resident / p.groups), p.rows);
            const dim3 grid(static_cast<unsigned>(each * p.groups));
            return threads <= 512 ? launch_pdl(norm_rows_kernel<kType, kIn, 512, 2>, grid, threads, stream, p)
                                  : launch_pdl(norm_rows_kernel<kType, kIn, 1024, 1>, grid, threads, stream, p);
        }
    const dim3 grid(static_cast<unsigned>(p.segments));
    if constexpr (!kInTurn)
        if (vecs == 2)
            return launch_pdl(norm_kernel<kType, kIn, 2, 0, 512, 3>, grid, threads, stream, p);
    return launch_pdl(norm_kernel<kType, kIn, kNormMaxVecs, 0, 1024, 1>, grid, threads, stream, p);
}

template <int kType>
cudaError_t launch_in(const NormParams &p, cudaStream_t stream)
{
    return p.residual ? launch<kType, kResidual>(p, stream)
           : p.gate   ? launch<kType, kGate>(p, stream)
                      : launch<kType, kPlain>(p, stream);
}

}  // namespace
}  // namespace ssd

extern "C" ssd_status_t ssd_rms_norm_fwd(
    void *y, float *scale, const void *x, void *residual, const void *gate, const float *weight,
    int64_t rows, int32_t dim, int32_t ngroups, int32_t out_type, float eps, int64_t y_stride,
    int64_t x_stride, int64_t residual_stride, int64_t gate_stride, ssd_stream_t stream)
{
    using namespace ssd;
    if (rows < 0 || dim <= 0 || ngroups <= 0 || dim % ngroups != 0 || !(eps >= 0x1p-80f && eps <= 1.f))
        return SSD_ERR_INVALID_ARG;
    if (out_type != SSD_KV_BF16 && out_type != SSD_KV_FP8_E4M3 && out_type != SSD_KV_INT8)
        return SSD_ERR_INVALID_ARG;
    const int32_t cols = dim / ngroups;
    if (cols % 8 != 0 || cols > 8 * 1024 * kNormMaxVecs || rows > INT32_MAX / 2 ||
        rows * ngroups > INT32_MAX / 2)
        return SSD_ERR_UNSUPPORTED;
    if (!kv_pitch(&y_stride, dim) || !kv_pitch(&x_stride, dim) || !kv_pitch(&residual_stride, dim) ||
        !kv_pitch(&gate_stride, dim))
        return SSD_ERR_INVALID_ARG;
    if (rows == 0)
        return SSD_OK;
    if (!y || !x || (out_type != SSD_KV_BF16) != (scale != nullptr) || (residual && gate))
        return SSD_ERR_INVALID_ARG;
    if (!kv_aligned16(y) || !kv_aligned16(x) || !kv_aligned16(residual) || !kv_aligned16(gate) ||
        !kv_aligned16(weight))
        return SSD_ERR_INVALID_ARG;
    const NormParams p = {y, scale, static_cast<const __nv_bfloat16 *>(x),
                          static_cast<const __nv_bfloat16 *>(gate), static_cast<__nv_bfloat16 *>(residual),
                          weight, rows, rows * ngroups, y_stride, x_stride, residual_stride, gate_stride,
                          ngroups, cols, eps};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = out_type == SSD_KV_BF16       ? launch_in<SSD_KV_BF16>(p, s)
                          : out_type == SSD_KV_FP8_E4M3 ? launch_in<SSD_KV_FP8_E4M3>(p, s)
                                                        : launch_in<SSD_KV_INT8>(p, s);
    return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}
