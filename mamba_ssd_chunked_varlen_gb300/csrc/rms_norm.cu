// Root-mean-square norm over groups of columns, with a residual's addition or a gate
// before it and an output in bf16 or in 8-bit codes:
//
//     s = x, x + residual (written back) or x silu(gate)
//     y = s w / sqrt(mean s^2 + eps);   codes: a = max|y|, code = round(y M / a), scale = a / M
//
// A segment is one row's group.  It is read once and stays in registers, eight values
// a load, between the sum of squares, the largest magnitude and the output: memory
// bounds it.
#include "layer_common.cuh"

namespace ssd {
namespace {

constexpr int kNormWarps = 4;        // segments of a CTA when a warp takes one
constexpr int kNormMaxVecs = 4;      // loads of eight values that a thread holds

enum NormInput { kPlain, kResidual, kGate };

struct NormParams {
    void *y;
    float *scale;
    const __nv_bfloat16 *x, *gate;
    __nv_bfloat16 *residual;
    const float *weight;
    int64_t segments, y_stride, x_stride, residual_stride, gate_stride;
    int32_t groups, cols;            // columns of a group
    float eps;
};

// Sum of v and largest of m over a segment's threads: a warp, or all of the CTA's.
template <bool kWarp>
__device__ __forceinline__ float segment_sum(float v, float *scratch)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (kWarp) {
        return v;
    } else {
        const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        if (lane == 0)
            scratch[threadIdx.x >> 5] = v;
        __syncthreads();
        v = lane < warps ? scratch[lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
}

template <bool kWarp>
__device__ __forceinline__ uint32_t segment_max(uint32_t v, uint32_t *scratch)
{
    v = __reduce_max_sync(0xffffffffu, v);
    if constexpr (kWarp) {
        return v;
    } else {
        const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        if (lane == 0)
            scratch[threadIdx.x >> 5] = v;
        __syncthreads();
        return __reduce_max_sync(0xffffffffu, lane < warps ? scratch[lane] : 0u);
    }
}

template <int kType, int kIn, int kVecs, bool kWarp>
__global__ void __launch_bounds__(kWarp ? kNormWarps * 32 : 1024) norm_kernel(const __grid_constant__ NormParams p)
{
    __shared__ float s_sum[2][32];
    __shared__ uint32_t s_max[32];
    const int tid = kWarp ? threadIdx.x & 31 : threadIdx.x, step = (kWarp ? 32 : blockDim.x) * 8;
    const int64_t seg = kWarp ? static_cast<int64_t>(blockIdx.x) * kNormWarps + (threadIdx.x >> 5) : blockIdx.x;
    pdl_wait();
    if (kWarp && seg >= p.segments)
        return;
    const int64_t row = seg / p.groups;
    const int col0 = static_cast<int>(seg % p.groups) * p.cols;
    float s[kVecs][8];
    uint4 raw[kVecs], other[kVecs];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        const int c = v * step + tid * 8;
        raw[v] = other[v] = make_uint4(0, 0, 0, 0);
        if (c < p.cols) {
            raw[v] = *reinterpret_cast<const uint4 *>(p.x + row * p.x_stride + col0 + c);
            if constexpr (kIn == kResidual)
                other[v] = *reinterpret_cast<const uint4 *>(p.residual + row * p.residual_stride + col0 + c);
            if constexpr (kIn == kGate)
                other[v] = *reinterpret_cast<const uint4 *>(p.gate + row * p.gate_stride + col0 + c);
        }
    }
    float sum = 0.f;
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
            if (c < p.cols)
                *reinterpret_cast<uint4 *>(p.residual + row * p.residual_stride + col0 + c) = round8(s[v]);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            sum = fmaf(s[v][k], s[v][k], sum);
    }
    sum = segment_sum<kWarp>(sum, s_sum[0]);
    float r = rsqrtf(sum / static_cast<float>(p.cols) + p.eps);
    if (!(sum < __int_as_float(0x7f800000))) {
        // squares out of range (or infinities and NaN): once more on s 2^-80, where eps is
        // nothing beside the mean
        sum = 0.f;
#pragma unroll
        for (int v = 0; v < kVecs; ++v)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                s[v][k] *= 0x1p-80f;
                sum = fmaf(s[v][k], s[v][k], sum);
            }
        sum = segment_sum<kWarp>(sum, s_sum[1]);
        r = rsqrtf(sum / static_cast<float>(p.cols));
    }
    uint32_t top = 0;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        const int c = v * step + tid * 8;
        float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
        if (p.weight && c < p.cols) {
            *reinterpret_cast<float4 *>(w) = __ldg(reinterpret_cast<const float4 *>(p.weight + col0 + c));
            *reinterpret_cast<float4 *>(w + 4) = __ldg(reinterpret_cast<const float4 *>(p.weight + col0 + c + 4));
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            s[v][k] = s[v][k] * r * w[k];
            if constexpr (kType != SSD_KV_BF16)
                top = max(top, c < p.cols ? __float_as_uint(s[v][k]) & 0x7fffffffu : 0u);
        }
        if constexpr (kType == SSD_KV_BF16) {
            if (c < p.cols)
                *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.y) + row * p.y_stride + col0 + c) =
                    round8(s[v]);
        }
    }
    if constexpr (kType != SSD_KV_BF16) {
        constexpr float kTop = kType == SSD_KV_INT8 ? kInt8Max : kE4m3Max;
        top = segment_max<kWarp>(top, s_max);
        const bool bad = top >= 0x7f800000u;
        const float a = fmaxf(__uint_as_float(top), kKvTiny);
        const float inv = __fdiv_rn(kTop, a);
        if (tid == 0)
            p.scale[seg] = bad ? __int_as_float(0x7fffffff) : __fdiv_rn(a, kTop);
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            const int c = v * step + tid * 8;
            if (c < p.cols)
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.y) + row * p.y_stride + col0 + c) =
                    bad ? make_uint2(0, 0) : encode8<kType>(s[v], inv);
        }
    }
}

template <int kType, int kIn>
cudaError_t launch(const NormParams &p, cudaStream_t stream)
{
    const int loads = p.cols / 8;
    // a warp a segment while its lanes hold four loads at most: no barrier
    if (loads <= 4 * 32) {
        const dim3 grid(static_cast<unsigned>((p.segments + kNormWarps - 1) / kNormWarps));
        return loads <= 32   ? launch_pdl(norm_kernel<kType, kIn, 1, true>, grid, kNormWarps * 32, stream, p)
               : loads <= 64 ? launch_pdl(norm_kernel<kType, kIn, 2, true>, grid, kNormWarps * 32, stream, p)
                             : launch_pdl(norm_kernel<kType, kIn, 4, true>, grid, kNormWarps * 32, stream, p);
    }
    const dim3 grid(static_cast<unsigned>(p.segments));
    const int vecs = loads <= 2 * 1024 ? 2 : kNormMaxVecs;
    const int threads = (loads + 32 * vecs - 1) / (32 * vecs) * 32;
    return vecs == 2 ? launch_pdl(norm_kernel<kType, kIn, 2, false>, grid, threads, stream, p)
                     : launch_pdl(norm_kernel<kType, kIn, kNormMaxVecs, false>, grid, threads, stream, p);
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
                          weight, rows * ngroups, y_stride, x_stride, residual_stride, gate_stride,
                          ngroups, cols, eps};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = out_type == SSD_KV_BF16       ? launch_in<SSD_KV_BF16>(p, s)
                          : out_type == SSD_KV_FP8_E4M3 ? launch_in<SSD_KV_FP8_E4M3>(p, s)
                                                        : launch_in<SSD_KV_INT8>(p, s);
    return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}
