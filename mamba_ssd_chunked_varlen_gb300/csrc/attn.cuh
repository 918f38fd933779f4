// Attention over the paged cache: launch parameters, workspace and work split.
#pragma once

#include <cuda.h>

#include "attn_common.cuh"
#include "ssd_device.cuh"

namespace ssd {

// One CTA per SM of a GB300; the work is split over exactly this many.
constexpr int kAttnCtas = 152;
constexpr int kTileKeys = 128;    // keys of a tile
constexpr int kTileRows = 128;    // query rows of a tile: whole tokens, each with
                                  // the query heads of one kv head

// A unit: up to two tiles of query rows of one sequence, with the range of key
// tiles that any of its rows sees.  A unit is worked on once per kv head.
struct alignas(32) AttnUnit {
    int32_t seq, row0, tokens;    // its new tokens: rows [row0, row0 + tokens)
    int32_t pos0;                 // position of the first (negative: padding)
    int32_t tile0, tiles;         // key tiles [tile0, tile0 + tiles), at least one
    int32_t kv_len;
    int32_t pad;
};
static_assert(sizeof(AttnUnit) == 32, "unit size");

struct AttnHeader {
    int64_t total;                // key tiles of all units and kv heads
    int32_t units;
    int32_t pad[61];
};
static_assert(sizeof(AttnHeader) == 256, "header size");

// The key tiles of all (unit, kv head) pairs, unit by unit and head by head,
// form one line that is cut into kAttnCtas equal pieces.  A pair that falls
// into several pieces leaves partial results, at most two per piece.
struct AttnParams {
    KvView c;
    __nv_bfloat16 *o;
    const __nv_bfloat16 *q;
    float *lse;                   // may be null
    int64_t o_stride;
    int32_t heads, group;         // query heads, of them per kv head
    int32_t tile_tokens;          // tokens of a tile: 128 / group
    int32_t window;
    float scale_log2;             // |softmax_scale| log2(e)
    int32_t negate;               // 1: softmax_scale < 0 (the scores change sign)
    AttnHeader *hdr;
    int32_t *seq_units;           // (batch + 1): units before each sequence
    AttnUnit *units;
    int64_t *cum;                 // (units + 1): key tiles before each unit, one head
    float *part_o;                // [2 kAttnCtas][256][dim]: sums of p v
    float2 *part_ml;              // [2 kAttnCtas][256]: maximum (log2), sum of p
};

struct AttnLayout {
    size_t header, seq_units, units, cum, part_ml, part_o, total;
};

inline int64_t attn_max_units(int64_t total_len, int32_t batch, int32_t group)
{
    const int64_t tokens = 2 * (kTileRows / group);
    return (total_len + tokens - 1) / tokens + batch;
}

inline AttnLayout attn_layout(int64_t total_len, int32_t batch, int32_t group, int32_t dim)
{
    const size_t units = static_cast<size_t>(attn_max_units(total_len, batch, group));
    AttnLayout L;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = (off + bytes + 255) & ~size_t(255);
        return at;
    };
    L.header = take(sizeof(AttnHeader));
    L.seq_units = take(sizeof(int32_t) * (static_cast<size_t>(batch) + 1));
    L.units = take(sizeof(AttnUnit) * units);
    L.cum = take(sizeof(int64_t) * (units + 1));
    L.part_ml = take(sizeof(float2) * 2 * kAttnCtas * 256);
    L.part_o = take(sizeof(float) * 2 * kAttnCtas * 256 * static_cast<size_t>(dim));
    L.total = off;
    return L;
}

// First tile of piece i of the line of `total` tiles, and the piece of tile t.
__host__ __device__ inline int64_t attn_piece_begin(int64_t total, int64_t i)
{
    return total * i / kAttnCtas;
}
__host__ __device__ inline int64_t attn_piece_of(int64_t total, int64_t t)
{
    return ((t + 1) * kAttnCtas + total - 1) / total - 1;
}

// Partial-result slot of a piece: its first segment (one that does not start
// its pair) or its last (one that does).
__device__ __forceinline__ int attn_slot(int64_t piece, bool starts)
{
    return static_cast<int>(2 * piece + (starts ? 1 : 0));
}

struct AttnMaps {
    CUtensorMap Q;       // bf16 (dim, heads, rows), box {64, group, tile_tokens}, 128-byte swizzle
    CUtensorMap K, V;    // bf16: (dim, page, pages * heads), box {64, min(page, 128), 1}, swizzled;
                         // 8-bit codes: bytes, box {dim, min(page, 128), 1}, packed
};

// The kernel of one cache type (one translation unit each).
cudaError_t launch_attn_bf16(const AttnParams &p, const AttnMaps &m, cudaStream_t s);
cudaError_t launch_attn_fp8(const AttnParams &p, const AttnMaps &m, cudaStream_t s);
cudaError_t launch_attn_int8(const AttnParams &p, const AttnMaps &m, cudaStream_t s);

}  // namespace ssd
