// Shared definitions of the layer operators (ssd_layers.h): the ragged batch with
// its slots as a kernel sees it, and rows of bf16.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/ssd_layers.h"
#include "attn_common.cuh"
#include "rows.cuh"
#include "ssd_device.cuh"

namespace ssd {

// The sequences and their pool slots, passed to kernels by value.
struct SlotBatch {
    const int32_t *qsl;          // (batch + 1)
    const uint8_t *has_init;     // (batch) or null
    const uint32_t *slots;       // (batch)
    uint32_t *errors;            // may be null
    int64_t total_len, max_slots;
    int32_t batch;
};

__device__ __forceinline__ void layer_error(uint32_t *errors, uint32_t flag)
{
    if (errors)
        atomicOr(errors, flag);
}

// Rows [begin, end) of sequence b; false (and the flag) when its bounds are none.
__device__ __forceinline__ bool seq_rows(const int32_t *qsl, int64_t total_len, uint32_t *errors, int b,
                                         int32_t &begin, int32_t &end)
{
    begin = qsl[b];
    end = qsl[b + 1];
    if (begin < 0 || end < begin || end > total_len || (b == 0 && begin != 0)) {
        layer_error(errors, SSD_DEVERR_BAD_QUERY_START_LOC);
        return false;
    }
    return true;
}

// The slot of sequence b, or -1 for none.
__device__ __forceinline__ int64_t seq_slot(const SlotBatch &s, int b)
{
    const uint32_t i = s.slots[b];
    if (static_cast<int64_t>(i) < s.max_slots)
        return i;
    if (i != SSD_NO_SLOT)
        layer_error(s.errors, SSD_DEVERR_BAD_CACHE_INDEX);
    return -1;
}

// The largest b with qsl[b] <= t (0 when there is none), by a whole warp: t the same
// in every lane, 32 probes at a time.
__device__ __forceinline__ int warp_last_start(const int32_t *qsl, int batch, int64_t t)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, n = batch;
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int at = lane * step;
        const uint32_t m = __ballot_sync(0xffffffffu, at < n && qsl[lo + at] <= t);
        const int k = m ? 31 - __clz(m) : 0;
        lo += k * step;
        n = min(step, n - k * step);
    }
    return lo;
}

// 1 / x, flushing results below 2^-126 to zero.
__device__ __forceinline__ float rcp_f32(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// v / (1 + e^-v).  (e^-v may overflow: v / infinity is the right zero.)
__device__ __forceinline__ float silu_f32(float v)
{
    return __fdividef(v, 1.f + __expf(-v));
}

// What every call with slots checks of them (total_len may be 0: slots are written all the same).
inline ssd_status_t slots_check(SlotBatch *s, const int32_t *qsl, const uint8_t *has_init,
                                const uint32_t *slots, int64_t total_len, int32_t batch,
                                int64_t max_slots, uint32_t *errors)
{
    if (total_len < 0 || batch < 0 || max_slots < 0)
        return SSD_ERR_INVALID_ARG;
    if (total_len > INT32_MAX / 2 || batch > INT32_MAX / 2)
        return SSD_ERR_UNSUPPORTED;
    if (batch > 0 && (!qsl || !slots))
        return SSD_ERR_INVALID_ARG;
    *s = SlotBatch{qsl, has_init, slots, errors, total_len, max_slots, batch};
    return SSD_OK;
}

}  // namespace ssd
