// Attention of units of few rows (at most 16: decoding sequences, a few proposed
// tokens), for one cache type and head_dim.
//
// Such a unit reads its whole context for a few rows: the reads bound it.  A
// 128-row tensor-core tile would be mostly empty, and its round trips through
// tensor memory take longer than the reads, so every warp works by itself on a
// piece of the line of 32-key tiles, with its own running maximum and sum, in
// registers.  (Tiles of the other kind from 9 rows on: 32 sequences of 15 rows 66 us
// instead of 58.)  Keys take the 16-row side of the products and query rows the
// 8-column side, so that eight rows (or twice eight) waste nothing (few_segment16: the
// other way round):
//
//   X = c (K Q^T),  m' = max(m, max X),  P = 2^(X - m'),  l = l 2^(m - m') + sum P,
//   O^T = O^T 2^(m - m') + V^T P
//
// (m moves only when X exceeds it by 8: P <= 2^8.)  The tensor pipes have time to
// spare, so P enters its product as two bf16, the rounded weight and what is left of
// it: with one, the output is off by half as much again as its own rounding.
//
// The keys come by asynchronous copies through shared memory, up to several tiles
// ahead and on into the next pair.  A lane copies exactly the bytes that its own
// fragments need, so a warp waits for nobody: with i = lane / 4, q = lane % 4, a
// lane has of K the pieces q, q + 4, ... (16 bytes each) of keys i and i + 8 of each
// sixteen, and of V, of their keys 2q, 2q + 1, 8 + 2q and 9 + 2q, the pieces i,
// i + 8, ...  Any order of a score's products serves as long as Q has the same, and a
// lane then holds neighbouring columns of the output.  Copies of keys past the
// context's end are filled with zeros, so nothing is read that no sequence owns.
//
// Measured, with 32 query heads on 8 kv heads of 128: 64 sequences of up to 8,192
// int8 keys, one token each: 137 us of the call's 149, for 639 MB, 4.7 TB/s, 69 % of the copy rate.  Each
// scheduler has three warps, which wait for one another's widening and products
// more than for memory (issue 51 %, integer pipe 56 %); more warps have too few
// registers (12 warps of 168: 152 us a call, 14 of 144: 179, 16 of 128: 162).  At
// head_dim 128 the 168 do not quite suffice either: some 60 (bf16) to 230 bytes
// a thread are spilled.  Tiles of 16 keys instead of 32: 160 us instead of 156.
//
// 8-bit codes are widened in registers, which is exact: K's to fp16 (the cheaper
// way; a row of Q is scaled by a power of two to fit fp16's range, exact but for
// elements below 2^-24 of the row's largest, which are off by 2^-32 of it at most), V's to
// bf16, because a weight times its key's scale needs the range.
#pragma once

#include <cfloat>

#include "attn_codes.cuh"

namespace ssd {
namespace {

constexpr float kFewRescale = 8.f;   // log2

template <int kType, int kDim>
struct FewCfg {
    static constexpr bool kQuant = kType != SSD_KV_BF16;
    static constexpr int kRowBytes = kQuant ? kDim : 2 * kDim;
    static constexpr int kLaneBytes = kRowBytes / 2;          // of 16 keys, a lane's 1 / 32
    static constexpr int kHalf = 32 * kLaneBytes;             // K or V of 16 keys
    static constexpr int kSlot = 2 * kHalf + (kQuant ? 128 : 0);   // K or V of a tile, with scales
    static constexpr int kSlots = kMaxSmemPerBlock / kFewWarps / kSlot;
    // the step that uses a K copies kSlots - 1 steps on: a K (0) or a V (1)
    static constexpr int kAhead = (kSlots - 1) % 2;
    static constexpr int kRing = kSlots * kSlot;              // bytes of a warp
    // a lane's copies: pieces of 16 bytes of two keys of K, of kVPiece bytes of four of V
    static constexpr int kKPieces = kLaneBytes / 32;
    static constexpr int kVPiece = kRowBytes >= 128 ? 16 : 8;
    static constexpr int kVPieces = kRowBytes / 8 / kVPiece;
    static constexpr int kBytes = kFewWarps * kRing;
};

// Puts the infinities and NaN of V into kN columns from d of a row's sums: those of the
// keys in [lo, hi) of tiles [ta, tb).  In tiles that some row does not see all of they were
// taken out; in the others they are in the sums, as NaN where an infinity met a weight's
// second part, so that sums that are not finite are looked up over all tiles.
template <int kDim, int kN>
__device__ __noinline__ void few_add_nonfinite(const AttnParams &p, const AttnUnit &e, int h, int ta,
                                               int tb, int hi, int lo, int d, float *acc)
{
    float found[kN];
    bool all = false;
    for (int k = 0; k < kN; ++k) {
        found[k] = 0.f;
        all = all || !(fabsf(acc[k]) <= FLT_MAX);
    }
    for (int t = ta; t < tb; ++t) {
        if (!all && !attn_partial(e, p.window, t * kFewKeys, kFewKeys, 0, e.tokens - 1))
            continue;
        for (int j = max(t * kFewKeys, max(lo, 0)); j < min((t + 1) * kFewKeys, hi); ++j) {
            const int64_t page = kv_page_of(p.c, e.seq, j);
            if (page < 0)
                continue;
            const __nv_bfloat16 *v =
                static_cast<const __nv_bfloat16 *>(p.c.v) + kv_row(p.c, page, h, j) * kDim + d;
            for (int k = 0; k < kN; ++k) {
                const float x = __bfloat162float(v[k]);
                if (!(fabsf(x) <= FLT_MAX))
                    found[k] += x;
            }
        }
    }
    for (int k = 0; k < kN; ++k)
        acc[k] = found[k] == 0.f ? acc[k] : found[k];
}

// The copies of a warp: tile by tile of its piece, K then V, slot by slot.
template <int kType, int kDim>
struct FewLoad {
    using C = FewCfg<kType, kDim>;
    const AttnParams &p;
    AttnWalk w;
    uint32_t dst0;               // shared-memory address of the warp's slots
    int put, t, ahead, my_page;  // slot's offset, tile; lane l has the page of the 16 keys from
                                 // tile t - ahead on + l
    bool there[2];               // of the tile's halves: whether they have a page,
    int64_t row[2];              // cache row of the first key
    uint32_t k_off, v_off;       // this lane's first piece in 16 keys of K and of V

    __device__ __forceinline__ FewLoad(const AttnParams &p_, int piece, uint32_t ring)
        : p(p_), w(p_.line[1], p_.c.heads, piece), dst0(ring), put(0), t(w.ta), ahead(32),
          my_page(-1), there{false, false}, row{0, 0}
    {
        const int lane = threadIdx.x & 31, i = lane >> 2, q = lane & 3;
        k_off = i * C::kRowBytes + q * 16;
        v_off = q * 2 * C::kRowBytes + i * C::kVPiece;
    }

    // The next tile's K (kV 0) or V (1), of which `left` keys are there.
    template <int kV>
    __device__ __forceinline__ void copy(int left)
    {
        const KvView &c = p.c;
        const int lane = threadIdx.x & 31, i = lane >> 2, q = lane & 3;
        constexpr int kKeys = kV ? 4 : 2, kPieces = kV ? C::kVPieces : C::kKPieces;
        constexpr int kPiece = kV ? C::kVPiece : 16, kNext = kV ? 8 * kPiece : 64;
        const uint8_t *cache = static_cast<const uint8_t *>(kV ? c.v : c.k) + (kV ? v_off : k_off);
        const uint32_t dst = dst0 + put + lane * kPiece;
        const int mine = kV ? q * 2 : i;
        if (left >= kFewKeys && there[0] && there[1]) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint8_t *src = cache + row[u] * C::kRowBytes;
#pragma unroll
                for (int n = 0; n < kKeys; ++n) {
                    const int key = kV ? (n & 1) + (n >> 1) * 8 : n * 8;
#pragma unroll
                    for (int k = 0; k < kPieces; ++k)
                        ptx::cp_async<kPiece>(dst + u * C::kHalf + (n * kPieces + k) * 32 * kPiece,
                                              src + key * C::kRowBytes + k * kNext, true);
                }
            }
        } else {
#pragma unroll 1
            for (int u = 0; u < 2; ++u) {
                const uint8_t *src = cache + (u ? row[1] : row[0]) * C::kRowBytes;
                const int keys = (u ? there[1] : there[0]) ? left - 16 * u : 0;
#pragma unroll 1
                for (int n = 0; n < kKeys; ++n) {
                    const int key = kV ? (n & 1) + (n >> 1) * 8 : n * 8;
#pragma unroll 1
                    for (int k = 0; k < kPieces; ++k)
                        ptx::cp_async<kPiece>(dst + u * C::kHalf + (n * kPieces + k) * 32 * kPiece,
                                              src + key * C::kRowBytes + k * kNext, mine + key < keys);
                }
            }
        }
        if constexpr (C::kQuant) {
            if (lane < 8)
                ptx::cp_async<16>(dst0 + put + 2 * C::kHalf + lane * 16,
                                  (kV ? c.v_scale : c.k_scale) + (lane < 4 ? row[0] : row[1]) + (lane & 3) * 4,
                                  lane < 4 ? there[0] && left > 0 : there[1] && left > 16);
        }
    }

    template <int kV>
    __device__ __forceinline__ void next()
    {
        const int lane = threadIdx.x & 31;
        if (w.more()) {
            const int j0 = (w.e.tile0 + t) * kFewKeys;
            if constexpr (kV == 0) {
                if (ahead == 32) {
                    ahead = 0;
                    const int j = j0 + lane * 16;
                    my_page = -1;
                    if (2 * t + lane < 2 * w.tb && j < w.e.kv_len)
                        my_page = static_cast<int>(kv_page_of(p.c, w.e.seq, j));
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int page = __shfl_sync(0xffffffffu, my_page, ahead + u);
                    there[u] = page >= 0;
                    row[u] = there[u] ? kv_row(p.c, page, w.h, j0 + 16 * u) : 0;
                }
                ahead += 2;
            }
            copy<kV>(w.e.kv_len - j0);
            if (kV && ++t == w.tb) {
                w.next();
                t = w.ta;
                ahead = 32;
            }
        }
        ptx::cp_async_commit();
        put = put + C::kSlot == C::kRing ? 0 : put + C::kSlot;
    }
};

// The fragments of query rows n 8 + i: element pairs in the order of K's pieces, and
// what turns a row's scores into log2 units.
template <int kType, int kDim, int kN>
__device__ __forceinline__ void few_query(const AttnParams &p, const AttnUnit &e, int h,
                                          uint32_t (&qb)[kN][kDim / 16][2], float (&unit)[kN])
{
    using C = FewCfg<kType, kDim>;
    const int lane = threadIdx.x & 31, i = lane >> 2, q = lane & 3;
    const int g = p.group, rows = e.tokens * g;
#pragma unroll
    for (int n = 0; n < kN; ++n) {
        const int row = n * 8 + i, tok = row / g;
        const uint4 *src = reinterpret_cast<const uint4 *>(
            p.q + (e.row0 + tok) * p.q_stride + static_cast<int64_t>(h * g + row % g) * kDim);
#pragma unroll
        for (int k = 0; k < kDim / 32; ++k) {
            // (eight elements, in the order of K's pieces)
            const int at = C::kQuant ? (k >> 1) * 8 + q * 2 + (k & 1) : k * 4 + q;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (row < rows)
                v = src[at];
            const uint32_t flip = p.negate ? 0x80008000u : 0u;
            qb[n][2 * k][0] = v.x ^ flip;
            qb[n][2 * k][1] = v.y ^ flip;
            qb[n][2 * k + 1][0] = v.z ^ flip;
            qb[n][2 * k + 1][1] = v.w ^ flip;
        }
        unit[n] = p.scale_log2;
        if constexpr (C::kQuant) {
            // the row's largest magnitude to [2^7, 2^8)
            float top = 0.f;
#pragma unroll
            for (int s = 0; s < kDim / 16; ++s)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    top = fmaxf(top, fmaxf(fabsf(__uint_as_float(qb[n][s][k] << 16)),
                                           fabsf(__uint_as_float(qb[n][s][k] & 0xffff0000u))));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int ex = static_cast<int>(__float_as_uint(top) >> 23);
            const int shift = ex == 0 || ex == 255 ? 0 : min(134 - ex, 100);
            const float up = pow2i(shift);
#pragma unroll
            for (int s = 0; s < kDim / 16; ++s)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const __half2 x = __floats2half2_rn(__uint_as_float(qb[n][s][k] << 16) * up,
                                                        __uint_as_float(qb[n][s][k] & 0xffff0000u) * up);
                    qb[n][s][k] = *reinterpret_cast<const uint32_t *>(&x);
                }
            unit[n] *= pow2i(-shift);
        }
    }
}

// A lane's values of piece k of sixteen keys: of keys 2q, 2q + 1, 8 + 2q and 9 + 2q.
template <int kType, int kDim, int kWords>
__device__ __forceinline__ void few_values(const uint8_t *half, int k, uint32_t (&v)[4][kWords])
{
    using C = FewCfg<kType, kDim>;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        const uint8_t *src = half + ((n * C::kVPieces + k) * 32 + lane) * C::kVPiece;
        if constexpr (kWords == 4) {
            const uint4 t4 = *reinterpret_cast<const uint4 *>(src);
            v[n][0] = t4.x;
            v[n][1] = t4.y;
            v[n][2] = t4.z;
            v[n][3] = t4.w;
        } else {
            const uint2 t2 = *reinterpret_cast<const uint2 *>(src);
            v[n][0] = t2.x;
            v[n][1] = t2.y;
        }
    }
}

// Takes infinities and NaN out: they would reach the rows that do not see them (0 times
// them), and are added at the end to those that do.  Whether there were any.
__device__ __forceinline__ bool few_clean(uint32_t (&v)[4][4])
{
    bool found = false;
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const bool a = (v[n][s] & 0x7f80u) == 0x7f80u;
            const bool b = (v[n][s] & 0x7f800000u) == 0x7f800000u;
            found = found || a || b;
            v[n][s] &= (a ? 0xffff0000u : 0xffffffffu) & (b ? 0xffffu : 0xffffffffu);
        }
    return found;
}

// Where a row of a segment goes: to the output, or to the piece's partial results.
struct FewRow {
    int64_t grow, prow;
    int tok, head;
    float m, l, inv;

    __device__ __forceinline__ FewRow(const AttnParams &p, const AttnWalk &w, int piece, int row, float m_,
                                      float l_)
        : prow(attn_slot(piece, w.starts()) * static_cast<int64_t>(kFewRows) + row), tok(row / p.group),
          head(w.h * p.group + row % p.group), m(m_), l(l_), inv(l > 0.f || l != l ? 1.f / l : 0.f)
    {
        grow = w.e.row0 + tok;
    }
    // Of eight columns from d on, infinities and NaN as the definition has them (a row
    // whose probabilities are NaN is NaN whatever its sums are).
    template <int kDim>
    __device__ __forceinline__ void add_nonfinite(const AttnParams &p, const AttnWalk &w, bool clean, int d,
                                                  float (&v)[8]) const
    {
        float most = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            most += fabsf(v[k]);     // (one that is not finite shows)
        if ((clean && most <= FLT_MAX) || l != l)
            return;
        const int pos = w.e.pos0 + tok;
        few_add_nonfinite<kDim, 8>(p, w.e, w.h, w.e.tile0 + w.ta, w.e.tile0 + w.tb, pos + 1,
                                   p.window > 0 ? pos - p.window + 1 : 0, d, v);
    }
    // eight columns from d on
    template <int kDim>
    __device__ __forceinline__ void store(const AttnParams &p, const AttnWalk &w, int d,
                                          const float (&v)[8]) const
    {
        if (w.whole()) {
            *reinterpret_cast<uint4 *>(p.o + grow * p.o_stride + static_cast<int64_t>(head) * kDim + d) =
                make_uint4(pack_bf16(v[0] * inv, v[1] * inv), pack_bf16(v[2] * inv, v[3] * inv),
                           pack_bf16(v[4] * inv, v[5] * inv), pack_bf16(v[6] * inv, v[7] * inv));
        } else {
            float4 *dst = reinterpret_cast<float4 *>(p.line[1].part_o + prow * kDim + d);
            dst[0] = make_float4(v[0], v[1], v[2], v[3]);
            dst[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
    }
    __device__ __forceinline__ void statistics(const AttnParams &p, const AttnWalk &w) const
    {
        if (!w.whole())
            p.line[1].part_ml[prow] = make_float2(m, l);
        else if (p.lse)
            p.lse[grow * p.heads + head] = l == 0.f ? -INFINITY : (log2f(l) + m) * 0.6931471805599453f;
    }
};

// One segment, with 8 kN rows (kN 2 for 8-bit caches alone, see few_segment16).
template <int kType, int kDim, int kN>
__device__ __forceinline__ void few_segment(const AttnParams &p, const AttnWalk &w, int piece,
                                            const uint8_t *slots, int &got, FewLoad<kType, kDim> &load)
{
    using C = FewCfg<kType, kDim>;
    const int lane = threadIdx.x & 31, i = lane >> 2, q = lane & 3;
    const AttnUnit &e = w.e;
    const int g = p.group, rows = e.tokens * g;
    const float c2 = p.scale_log2;
    uint32_t qb[kN][kDim / 16][2];
    float unit[kN], cr[kN][2];   // (a lane's scores are of rows 2q and 2q + 1)
    few_query<kType, kDim, kN>(p, e, w.h, qb, unit);
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r)
            cr[n][r] = __shfl_sync(0xffffffffu, unit[n], (q * 2 + r) * 4);
    float o[kN][kDim / 16][4];
    // -m: the reference begins with the least finite number, which is one like any other
    float nm[kN][2], l[kN][2];
#pragma unroll
    for (int n = 0; n < kN; ++n) {
#pragma unroll
        for (int s = 0; s < kDim / 16; ++s)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                o[n][s][k] = 0.f;
        nm[n][0] = nm[n][1] = FLT_MAX;
        l[n][0] = l[n][1] = 0.f;
    }
    bool nonfinite = false;

    for (int t = w.ta; t < w.tb; ++t) {
        const int j0 = (e.tile0 + t) * kFewKeys;
        const bool hides = attn_partial(e, p.window, j0, kFewKeys, 0, e.tokens - 1);
        // ---- scores: keys i, i + 8, ... (k), rows 2q and 2q + 1 of each eight ----
        ptx::cp_async_wait<C::kSlots - 2>();
        __syncwarp();                            // the other lanes' copies of the scales
        const uint8_t *slot = slots + got;
        got = got + C::kSlot == C::kRing ? 0 : got + C::kSlot;
        load.template next<C::kAhead>();
        float x[2][kN][4];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    x[u][n][k] = 0.f;
#pragma unroll
        for (int k = 0; k < C::kKPieces; ++k)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint8_t *src = slot + u * C::kHalf + (k * 32 + lane) * 16;
                const uint4 va = *reinterpret_cast<const uint4 *>(src);
                const uint4 vb = *reinterpret_cast<const uint4 *>(src + C::kKPieces * 512);
                const uint32_t a4[4] = {va.x, va.y, va.z, va.w}, b4[4] = {vb.x, vb.y, vb.z, vb.w};
                if constexpr (C::kQuant) {
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        uint32_t a[2], b[2];
                        half4<kType>(a4[s], a);
                        half4<kType>(b4[s], b);
                        const uint32_t f[4] = {a[0], b[0], a[1], b[1]};
#pragma unroll
                        for (int n = 0; n < kN; ++n)
                            ptx::mma_16816_f16(x[u][n], f, qb[n][k * 4 + s][0], qb[n][k * 4 + s][1]);
                    }
                } else {
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const uint32_t f[4] = {a4[2 * s], b4[2 * s], a4[2 * s + 1], b4[2 * s + 1]};
#pragma unroll
                        for (int n = 0; n < kN; ++n)
                            ptx::mma_16816(x[u][n], f, qb[n][k * 2 + s][0], qb[n][k * 2 + s][1]);
                    }
                }
            }
        const float *scales = reinterpret_cast<const float *>(slot + 2 * C::kHalf) + i;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float ks = 1.f;
            if constexpr (C::kQuant)
                ks = scales[8 * k];
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    x[k / 2][n][k % 2 * 2 + r] *= C::kQuant ? ks * cr[n][r] : c2;
        }
        uint32_t unseen = 0;     // a bit per score of the lane
        if (hides) {
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int pos = e.pos0 + min((n * 8 + q * 2 + r) / g, e.tokens - 1);
                    const int lo = p.window > 0 ? pos - p.window + 1 : INT32_MIN / 2;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int j = j0 + i + k * 8;
                        if (j < lo || j > pos) {
                            x[k / 2][n][k % 2 * 2 + r] = -INFINITY;
                            unseen |= 1u << ((k * kN + n) * 2 + r);
                        }
                    }
                }
        }
        // ---- probabilities ----
        auto largest = [&](int n, int r) {
            return fmaxf(fmaxf(x[0][n][r], x[0][n][2 + r]), fmaxf(x[1][n][r], x[1][n][2 + r]));
        };
        float over = -INFINITY;
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r)
                over = fmaxf(over, largest(n, r) + nm[n][r]);
        if (__any_sync(0xffffffffu, over > kFewRescale)) {
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float v = largest(n, r);
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                    const float to = fminf(nm[n][r], -v);
                    const float f = to == nm[n][r] ? 1.f : ptx::ex2(to - nm[n][r]);
                    nm[n][r] = to;
                    l[n][r] *= f;
#pragma unroll
                    for (int s = 0; s < kDim / 16; ++s) {
                        o[n][s][r] *= f;
                        o[n][s][2 + r] *= f;
                    }
                }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float &v = x[u][n][k];
                    v = ptx::ex2(v + nm[n][k & 1]);
                    l[n][k & 1] += v;
                }
        // ---- V^T P ----
        ptx::cp_async_wait<C::kSlots - 2>();
        __syncwarp();
        slot = slots + got;
        got = got + C::kSlot == C::kRing ? 0 : got + C::kSlot;
        load.template next<1 - C::kAhead>();
        if constexpr (C::kQuant) {
            scales = reinterpret_cast<const float *>(slot + 2 * C::kHalf) + i;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float vs = scales[8 * k];
#pragma unroll
                for (int n = 0; n < kN; ++n)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        // (a hidden key's scale may be NaN)
                        float &w = x[k / 2][n][k % 2 * 2 + r];
                        w = unseen >> ((k * kN + n) * 2 + r) & 1 ? 0.f : w * vs;
                    }
            }
        }
        uint32_t pb[2][kN][2], pl[2][kN][2];     // the weights as two bf16 each
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int n = 0; n < kN; ++n) {
                const float a = x[k / 2][n][k % 2 * 2], b = x[k / 2][n][k % 2 * 2 + 1];
                const uint32_t top = pack_bf16(a, b);
                pb[k / 2][n][k % 2] = ptx::transpose8(top);
                pl[k / 2][n][k % 2] = ptx::transpose8(pack_bf16(
                    a - __uint_as_float(top << 16), b - __uint_as_float(top & 0xffff0000u)));
            }
#pragma unroll
        for (int k = 0; k < C::kVPieces; ++k)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                constexpr int kWords = C::kVPiece / 4;
                uint32_t v[4][kWords];
                few_values<kType, kDim>(slot + u * C::kHalf, k, v);
                if constexpr (C::kQuant) {
#pragma unroll
                    for (int s = 0; s < kWords; ++s) {
                        uint32_t a[4], b[4];
                        widen_columns<kType, 0>(v[0][s], v[1][s], a);
                        widen_columns<kType, 2>(v[0][s], v[1][s], a + 2);
                        widen_columns<kType, 0>(v[2][s], v[3][s], b);
                        widen_columns<kType, 2>(v[2][s], v[3][s], b + 2);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t f[4] = {a[2 * j], a[2 * j + 1], b[2 * j], b[2 * j + 1]};
#pragma unroll
                            for (int n = 0; n < kN; ++n) {
                                ptx::mma_16816(o[n][s * 2 + j], f, pb[u][n][0], pb[u][n][1]);
                                ptx::mma_16816(o[n][s * 2 + j], f, pl[u][n][0], pl[u][n][1]);
                            }
                        }
                    }
                } else {
                    if (hides)
                        nonfinite = few_clean(v) || nonfinite;
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const uint32_t f[4] = {
                            __byte_perm(v[0][s], v[1][s], 0x5410), __byte_perm(v[0][s], v[1][s], 0x7632),
                            __byte_perm(v[2][s], v[3][s], 0x5410), __byte_perm(v[2][s], v[3][s], 0x7632)};
#pragma unroll
                        for (int n = 0; n < kN; ++n) {
                            ptx::mma_16816(o[n][k * 4 + s], f, pb[u][n][0], pb[u][n][1]);
                            ptx::mma_16816(o[n][k * 4 + s], f, pl[u][n][0], pl[u][n][1]);
                        }
                    }
                }
            }
    }

    // ---- output: rows 2q and 2q + 1 of each eight, the lane's columns ----
    const bool clean = !__any_sync(0xffffffffu, nonfinite);
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[n][r] += __shfl_xor_sync(0xffffffffu, l[n][r], 4);
            l[n][r] += __shfl_xor_sync(0xffffffffu, l[n][r], 8);
            l[n][r] += __shfl_xor_sync(0xffffffffu, l[n][r], 16);
            const int row = n * 8 + q * 2 + r;
            if (row >= rows)
                continue;
            const FewRow out(p, w, piece, row, -nm[n][r], l[n][r]);
            // runs of eight neighbouring columns: products s .. s + 3 with both of theirs
#pragma unroll
            for (int s = 0; s < kDim / 16; s += 4) {
                const int d = C::kQuant ? i * (kDim / 8) + s * 2 : s * 16 + i * 8;
                float v[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    v[2 * k] = o[n][s + k][r];
                    v[2 * k + 1] = o[n][s + k][2 + r];
                }
                if constexpr (!C::kQuant)
                    out.add_nonfinite<kDim>(p, w, clean, d, v);
                out.store<kDim>(p, w, d, v);
            }
            if (i == 0)
                out.statistics(p, w);
        }
}

// One segment of a bf16 cache with 9 to 16 rows: query rows take the 16-row side, keys
// the 8-column side, so that the scores' fragments are the weights' without a transpose
// (32 sequences of 15 rows: 51.5 us, with few_segment 53.0.  For 8-bit caches its
// registers do not suffice beside what widens the codes, and cost the units of fewer
// rows as well: 64 sequences decoding 149 us -> 163).
template <int kDim>
__device__ __forceinline__ void few_segment16(const AttnParams &p, const AttnWalk &w, int piece,
                                              const uint8_t *slots, int &got,
                                              FewLoad<SSD_KV_BF16, kDim> &load)
{
    using C = FewCfg<SSD_KV_BF16, kDim>;
    const int lane = threadIdx.x & 31, i = lane >> 2, q = lane & 3;
    const AttnUnit &e = w.e;
    const int g = p.group, rows = e.tokens * g;
    uint32_t qb[2][kDim / 16][2];
    float unit[2];               // (of rows i and i + 8: the scale)
    few_query<SSD_KV_BF16, kDim, 2>(p, e, w.h, qb, unit);
    // product 8 k + t: columns 8 (8 k + n) + t, n its column
    float o[kDim / 8][4];
    float nm[2], l[2];           // (see few_segment)
#pragma unroll
    for (int t = 0; t < kDim / 8; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            o[t][k] = 0.f;
    nm[0] = nm[1] = FLT_MAX;
    l[0] = l[1] = 0.f;
    bool nonfinite = false;

    for (int t = w.ta; t < w.tb; ++t) {
        const int j0 = (e.tile0 + t) * kFewKeys;
        const bool hides = attn_partial(e, p.window, j0, kFewKeys, 0, e.tokens - 1);
        // ---- scores of eight keys each: rows i and i + 8, keys 2q and 2q + 1 ----
        ptx::cp_async_wait<C::kSlots - 2>();
        __syncwarp();
        const uint8_t *slot = slots + got;
        got = got + C::kSlot == C::kRing ? 0 : got + C::kSlot;
        load.template next<C::kAhead>();
        float x[4][4];           // [eight keys][row i: two keys, row i + 8: two keys]
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                x[k][r] = 0.f;
#pragma unroll
        for (int k = 0; k < C::kKPieces; ++k)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint4 v = *reinterpret_cast<const uint4 *>(
                    slot + u / 2 * C::kHalf + ((u % 2 * C::kKPieces + k) * 32 + lane) * 16);
                const uint32_t v4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const uint32_t(&a)[2] = qb[0][k * 2 + s], (&b)[2] = qb[1][k * 2 + s];
                    const uint32_t rows4[4] = {a[0], b[0], a[1], b[1]};
                    ptx::mma_16816(x[u], rows4, v4[2 * s], v4[2 * s + 1]);
                }
            }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                x[k][r] *= unit[r / 2];
        if (hides) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int pos = e.pos0 + min((r * 8 + i) / g, e.tokens - 1);
                const int lo = p.window > 0 ? pos - p.window + 1 : INT32_MIN / 2;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int j = j0 + k / 2 * 8 + 2 * q + k % 2;
                    if (j < lo || j > pos)
                        x[k / 2][2 * r + k % 2] = -INFINITY;
                }
            }
        }
        // ---- probabilities ----
        auto largest = [&](int r) {
            float v = fmaxf(x[0][2 * r], x[0][2 * r + 1]);
#pragma unroll
            for (int k = 1; k < 4; ++k)
                v = fmaxf(v, fmaxf(x[k][2 * r], x[k][2 * r + 1]));
            return v;
        };
        if (__any_sync(0xffffffffu, fmaxf(largest(0) + nm[0], largest(1) + nm[1]) > kFewRescale)) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float v = largest(r);
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
                const float to = fminf(nm[r], -v);
                const float f = to == nm[r] ? 1.f : ptx::ex2(to - nm[r]);
                nm[r] = to;
                l[r] *= f;
#pragma unroll
                for (int s = 0; s < kDim / 8; ++s) {
                    o[s][2 * r] *= f;
                    o[s][2 * r + 1] *= f;
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                x[k][r] = ptx::ex2(x[k][r] + nm[r / 2]);
                l[r / 2] += x[k][r];
            }
        // ---- P V ----
        ptx::cp_async_wait<C::kSlots - 2>();
        __syncwarp();
        slot = slots + got;
        got = got + C::kSlot == C::kRing ? 0 : got + C::kSlot;
        load.template next<1 - C::kAhead>();
        uint32_t pa[2][4], pl[2][4];             // the weights as two bf16 each
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float a = x[k][2 * r], b = x[k][2 * r + 1];
                const uint32_t top = pack_bf16(a, b);
                pa[k / 2][k % 2 * 2 + r] = top;
                pl[k / 2][k % 2 * 2 + r] =
                    pack_bf16(a - __uint_as_float(top << 16), b - __uint_as_float(top & 0xffff0000u));
            }
#pragma unroll
        for (int k = 0; k < C::kVPieces; ++k)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                uint32_t v[4][4];
                few_values<SSD_KV_BF16, kDim>(slot + u * C::kHalf, k, v);
                if (hides)
                    nonfinite = few_clean(v) || nonfinite;
                auto product = [&](int s, uint32_t b0, uint32_t b1) {
                    ptx::mma_16816(o[s], pa[u], b0, b1);
                    ptx::mma_16816(o[s], pl[u], b0, b1);
                };
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    product(k * 8 + 2 * s, __byte_perm(v[0][s], v[1][s], 0x5410),
                            __byte_perm(v[2][s], v[3][s], 0x5410));
                    product(k * 8 + 2 * s + 1, __byte_perm(v[0][s], v[1][s], 0x7632),
                            __byte_perm(v[2][s], v[3][s], 0x7632));
                }
            }
    }

    // ---- output: rows i and i + 8, runs of eight neighbouring columns ----
    const bool clean = !__any_sync(0xffffffffu, nonfinite);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        const int row = r * 8 + i;
        if (row >= rows)
            continue;
        const FewRow out(p, w, piece, row, -nm[r], l[r]);
#pragma unroll
        for (int s = 0; s < kDim / 8; s += 8)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int d = (s + 2 * q + c) * 8;
                float v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    v[k] = o[s + k][2 * r + c];
                out.add_nonfinite<kDim>(p, w, clean, d, v);
                out.store<kDim>(p, w, d, v);
            }
        if (q == 0)
            out.statistics(p, w);
    }
}

template <int kType, int kDim>
__global__ void __launch_bounds__(kFewWarps * 32, 1)
    attn_few_kernel(const __grid_constant__ AttnParams p)
{
    using C = FewCfg<kType, kDim>;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5;
    const int piece = blockIdx.x + warp * kAttnCtas;    // short lines: a piece per CTA first
    pdl_launch_dependents();
    // the plan (behind the tiles' kernel the plan's grid has long ended, but only this
    // grid's own wait makes its writes visible here)
    pdl_wait();
    const uint8_t *slots = smem + warp * C::kRing;
    FewLoad<kType, kDim> load(p, piece, ptx::smem_u32(slots));
    if (load.w.more()) {
        AttnWalk w = load.w;
        int got = 0;
#pragma unroll 1
        for (int k = 0; k < (C::kSlots - 1) / 2; ++k) {
            load.template next<0>();
            load.template next<1>();
        }
        if constexpr (C::kAhead == 1)
            load.template next<0>();
        for (; w.more(); w.next()) {
            if (w.e.tokens * p.group <= 8)
                few_segment<kType, kDim, 1>(p, w, piece, slots, got, load);
            else if constexpr (C::kQuant)
                few_segment<kType, kDim, 2>(p, w, piece, slots, got, load);
            else
                few_segment16<kDim>(p, w, piece, slots, got, load);
        }
        ptx::cp_async_wait<0>();
    }
}

template <int kType, int kDim>
cudaError_t launch_few_one(const AttnParams &p, cudaStream_t stream)
{
    using C = FewCfg<kType, kDim>;
    static_assert(C::kBytes <= kMaxSmemPerBlock && C::kSlots >= 2, "shared memory");
    static SmemOptIn opted;
    cudaError_t e =
        ensure_max_smem(reinterpret_cast<const void *>(attn_few_kernel<kType, kDim>), opted);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kAttnCtas);
    cfg.blockDim = dim3(kFewWarps * 32);
    cfg.dynamicSmemBytes = C::kBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_few_kernel<kType, kDim>, p);
}

template <int kType>
cudaError_t launch_few(const AttnParams &p, cudaStream_t stream)
{
    return p.c.dim == 128 ? launch_few_one<kType, 128>(p, stream) : launch_few_one<kType, 64>(p, stream);
}

}  // namespace
}  // namespace ssd
