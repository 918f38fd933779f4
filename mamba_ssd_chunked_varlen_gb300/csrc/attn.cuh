// Attention over the paged cache: launch parameters, workspace and work split.
#pragma once

#include <cuda.h>

#include "attn_common.cuh"
#include "ssd_device.cuh"

namespace ssd {

// One CTA per SM of a GB300.
constexpr int kAttnCtas = 152;
constexpr int kTileKeys = 128;    // keys of a tile
constexpr int kTileRows = 128;    // query rows of a tile: whole tokens, each with
                                  // the query heads of one kv head

constexpr int kFewRows = 16;      // most query rows of a unit of the kind "few"
constexpr int kFewKeys = 32;      // keys of such a unit's tile
constexpr int kFewWarps = 12;     // warps of a CTA of its kernel

// A unit: query rows of one sequence with the range of key tiles that any of its
// rows sees.  A unit is worked on once per kv head.  Kind 0: up to two tiles of
// rows, for the tensor cores; kind 1: at most kFewRows rows (attn_few.cuh).
struct alignas(32) AttnUnit {
    int32_t seq, row0, tokens;    // its new tokens: rows [row0, row0 + tokens)
    int32_t pos0;                 // position of the first (negative: padding)
    int32_t tile0, tiles;         // key tiles of its kind [tile0, tile0 + tiles), at least one
    int32_t kv_len;
    int32_t pad;
};
static_assert(sizeof(AttnUnit) == 32, "unit size");

// The key tiles of all (unit, kv head) pairs of one kind, unit by unit and head
// by head, form a line that is cut into equal pieces: a piece per CTA (kind 0), or
// per warp (kind 1; fewer pieces when the line is short).  A pair that falls
// into several pieces leaves partial results, at most two per piece.
struct alignas(32) AttnPiece {
    int32_t tiles;                // its tiles of the line, none past the last piece
    int32_t u, h, ta;             // unit, kv head and tile of the unit where it begins
    int32_t pad[4];
    AttnUnit e;                   // the unit
};

struct AttnLine {
    const AttnUnit *units;
    const AttnPiece *pieces;
    int64_t *cum;                 // (units): key tiles before each unit, one head (the plan's)
    float *part_o;                // sums of p v: few [2 pieces][rows][dim], tiles
                                  // [2 pieces][dim / 4][rows][4]
    float2 *part_ml;              // [2 pieces][rows]: reference (log2), sum of p
    int4 *split;                  // [pieces] of a piece that begins within a pair begun by the
                                  // one before: {row0, tokens + (kv head << 9), that piece, the
                                  // pair's last}; zeros otherwise
};

// Most pieces of each kind, and the pieces of a line of `total` tiles.  A short line
// gets as few as leave the longest as short as it can be, because partial results
// cost more than shorter pieces among them save (24 sequences, 2,900 tiles of few rows:
// pieces of two 70.2 us, of one and two 72.2).  A long one gets them all: warps left
// over would be missed (64 sequences decoding: 151.5 us, with the same rule 155.7).
__host__ __device__ constexpr int attn_max_pieces(int kind)
{
    return kind ? kAttnCtas * kFewWarps : kAttnCtas;
}
__host__ __device__ inline int attn_pieces(int kind, int64_t total)
{
    const int most = attn_max_pieces(kind);
    const int64_t longest = (total + most - 1) / most;
    if (longest > 4)
        return most;
    return total > 0 ? static_cast<int>((total + longest - 1) / longest) : 0;
}

constexpr int kJoinWide = 128;    // pieces of a row that one warp of the join adds up

struct AttnParams {
    KvView c;
    __nv_bfloat16 *o;
    const __nv_bfloat16 *q;
    float *lse;                   // may be null
    int64_t o_stride, q_stride;
    int32_t heads, group;         // query heads, of them per kv head
    int32_t tile_tokens;          // tokens of a tile: 128 / group
    int32_t window;
    float scale_log2;             // |softmax_scale| log2(e)
    int32_t negate;               // 1: softmax_scale < 0 (the scores change sign)
    int32_t *seq_units;           // (batch): units before each sequence
    AttnLine line[2];
};

// Rows of a partial result of each kind.
__host__ __device__ constexpr int attn_part_rows(int kind) { return kind ? kFewRows : 2 * kTileRows; }

struct AttnLayout {
    size_t seq_units, units[2], pieces[2], cum[2], split[2], part_ml[2], part_o[2], total;
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
    L.seq_units = take(sizeof(int32_t) * (static_cast<size_t>(batch) + 1));
    for (int k = 0; k < 2; ++k) {
        const size_t rows = 2 * static_cast<size_t>(attn_max_pieces(k)) * attn_part_rows(k);
        L.units[k] = take(sizeof(AttnUnit) * units);
        L.pieces[k] = take(sizeof(AttnPiece) * static_cast<size_t>(attn_max_pieces(k)));
        L.cum[k] = take(sizeof(int64_t) * units);
        L.split[k] = take(sizeof(int4) * static_cast<size_t>(attn_max_pieces(k)));
        L.part_ml[k] = take(sizeof(float2) * rows);
        L.part_o[k] = take(sizeof(float) * rows * static_cast<size_t>(dim));
    }
    L.total = off;
    return L;
}

// Partial-result slot of a piece: its first segment (one that does not start
// its pair) or its last (one that does).
__device__ __forceinline__ int attn_slot(int64_t piece, bool starts)
{
    return static_cast<int>(2 * piece + (starts ? 1 : 0));
}

// A piece of a line, segment by segment: a segment is the part of one (unit, kv
// head) pair that lies in the piece.
struct AttnWalk {
    const AttnLine &line;
    int32_t heads;
    int32_t left;             // tiles of the piece from the segment's first on
    int32_t u, h, ta, tb;     // unit, kv head, tiles [ta, tb) of the unit's
    AttnUnit e;

    __device__ __forceinline__ AttnWalk(const AttnLine &l, int32_t heads_, int piece)
        : line(l), heads(heads_)
    {
        const AttnPiece pc = line.pieces[piece];
        left = pc.tiles;
        u = pc.u;
        h = pc.h;
        ta = pc.ta;
        e = pc.e;
        tb = min(ta + left, e.tiles);
    }
    __device__ __forceinline__ bool more() const { return left > 0; }
    __device__ __forceinline__ void next()
    {
        left -= tb - ta;
        if (left <= 0)
            return;
        ta = 0;
        if (++h == heads) {
            h = 0;
            e = line.units[++u];
        }
        tb = min(left, e.tiles);
    }
    // whether the segment begins its pair, and is all of it
    __device__ __forceinline__ bool starts() const { return ta == 0; }
    __device__ __forceinline__ bool whole() const { return ta == 0 && tb == e.tiles; }
};

// Whether some row of tokens [first, last] of a unit does not see all of the n
// keys from k0 on.
__device__ __forceinline__ bool attn_partial(const AttnUnit &e, int window, int k0, int n, int first,
                                             int last)
{
    return k0 + n > e.pos0 + first + 1 || (window > 0 && k0 < e.pos0 + last - window + 1);
}

struct AttnMaps {
    CUtensorMap Q;       // bf16 (dim, heads, rows), box {64, group, tile_tokens}, 128-byte swizzle
    CUtensorMap K, V;    // bf16: (dim, page, pages * heads), box {64, min(page, 128), 1}, swizzled;
                         // 8-bit codes: bytes, box {dim, min(page, 128), 1}, packed
};

// The two kernels of one cache type (one translation unit each).
cudaError_t launch_attn_bf16(const AttnParams &p, const AttnMaps &m, cudaStream_t s);
cudaError_t launch_attn_fp8(const AttnParams &p, const AttnMaps &m, cudaStream_t s);
cudaError_t launch_attn_int8(const AttnParams &p, const AttnMaps &m, cudaStream_t s);
cudaError_t launch_attn_few_bf16(const AttnParams &p, cudaStream_t s);
cudaError_t launch_attn_few_fp8(const AttnParams &p, cudaStream_t s);
cudaError_t launch_attn_few_int8(const AttnParams &p, cudaStream_t s);

}  // namespace ssd
