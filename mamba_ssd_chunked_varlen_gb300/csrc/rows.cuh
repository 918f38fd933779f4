// Rows of bf16 widened, and rounded to bf16 or to 8-bit codes, eight values at a time.
#pragma once

#include <cstdint>
#include <cuda_fp8.h>

#include "attn_common.cuh"
#include "ssd_device.cuh"

namespace ssd {

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

__device__ __forceinline__ uint4 round8(const float (&x)[8])
{
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                      pack_bf16(x[6], x[7]));
}

// Codes of x * inv: the nearest integers, or e4m3 numbers.
template <int kType>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv)
{
    uint32_t w[2] = {0u, 0u};
    if constexpr (kType == SSD_KV_INT8) {
        // added to 1.5 2^23, the nearest integer (ties to even) is in the low byte
        uint32_t y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            y[i] = __float_as_uint(__fadd_rn(__fmul_rn(x[i], inv), 12582912.f));
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = __byte_perm(__byte_perm(y[4 * i], y[4 * i + 1], 0x0040),
                               __byte_perm(y[4 * i + 2], y[4 * i + 3], 0x0040), 0x5410);
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

}  // namespace ssd
