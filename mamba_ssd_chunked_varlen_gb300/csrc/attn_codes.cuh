// Widening of 8-bit codes to bf16 pairs, for the attention kernels.
#pragma once

#include <cuda_fp16.h>

#include "attn.cuh"
#include "attn_ptx.cuh"
#include "kernels.cuh"

namespace ssd {
namespace {

// Codes to bf16 pairs (both exact).  int8: with the low seven bits put into
// bf16's mantissa at 128 = 0x4300, code = (128 + low7) - (128 or 256 with the sign bit).
__device__ __forceinline__ uint32_t int8_pair(uint32_t two)   // codes in bytes 0 and 2
{
    const uint32_t a = (two & 0x007f007fu) | 0x43004300u, b = (two & 0x00800080u) | 0x43004300u;
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The same with half the integer instructions and two for the FMA pipe: bf16's smallest
// numbers are multiples of 2^-133, so that code + 128 in the low byte is
// (code + 128) 2^-133; times 2^127, less 2, times 64.  (Tiles, whose softmax needs the
// integer pipe: 24 sequences 69.7 -> 68.0 us; few rows wait for results rather than
// slots: 64 sequences decoding 151.5 -> 152.9.)
__device__ __forceinline__ uint32_t int8_pair_fma(uint32_t plus128)   // bytes 1 and 3 zero
{
    uint32_t r;
    asm("{\n\t.reg .b32 t;\n\tfma.rn.bf16x2 t, %1, %2, %3;\n\tmul.rn.bf16x2 %0, t, %4;\n\t}"
        : "=r"(r)
        : "r"(plus128), "r"(0x7f007f00u), "r"(0xc000c000u), "r"(0x42804280u));
    return r;
}

template <int kType>
__device__ __forceinline__ void widen4(uint32_t codes, uint32_t *out)
{
    if constexpr (kType == SSD_KV_INT8) {
        const uint32_t u = codes ^ 0x80808080u;
        out[0] = int8_pair_fma(__byte_perm(u, 0, 0x4140));
        out[1] = int8_pair_fma(__byte_perm(u, 0, 0x4342));
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t h2;
            const uint16_t pair = static_cast<uint16_t>(codes >> (16 * i));
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(pair));
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h2));
            out[i] = pack_bf16(f.x, f.y);
        }
    }
}

// Codes to fp16 pairs (both exact): half the instructions of bf16, for products
// whose other operand is kept in fp16's range.  int8: code + 128 in the mantissa of
// 1024 = 0x6400, minus 1152.
__device__ __forceinline__ uint32_t int8_half(uint32_t plus1152)
{
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(plus1152), "r"(0x64806480u));
    return r;
}

__device__ __forceinline__ uint32_t e4m3_half(uint32_t two)   // codes in the low bytes
{
    uint32_t r;
    const uint16_t pair = static_cast<uint16_t>(two);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(pair));
    return r;
}

// Four codes to two pairs of neighbours.
template <int kType>
__device__ __forceinline__ void half4(uint32_t codes, uint32_t *out)
{
    if constexpr (kType == SSD_KV_INT8) {
        const uint32_t u = codes ^ 0x80808080u;
        out[0] = int8_half(__byte_perm(u, 0x64646464u, 0x4140));
        out[1] = int8_half(__byte_perm(u, 0x64646464u, 0x4342));
    } else {
        out[0] = e4m3_half(codes);
        out[1] = e4m3_half(codes >> 16);
    }
}

// Of two registers with codes of two keys, neighbouring columns in their bytes:
// the pairs (bf16) of the two keys' codes of columns b and b + 1 (b 0 or 2).
template <int kType, int b>
__device__ __forceinline__ void widen_columns(uint32_t key0, uint32_t key1, uint32_t *out)
{
    if constexpr (kType == SSD_KV_INT8) {
        const uint32_t x = __byte_perm(key0, key1, b ? 0x7632 : 0x5410);   // codes in bytes 0, 2 and 1, 3
        out[0] = int8_pair(x);
        out[1] = int8_pair(x >> 8);
    } else {
        widen4<kType>(__byte_perm(key0, key1, b ? 0x7362 : 0x5140), out);
    }
}

}  // namespace
}  // namespace ssd
