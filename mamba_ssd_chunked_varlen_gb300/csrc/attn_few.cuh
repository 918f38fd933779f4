// Attention of units of few rows (at most 32: decoding sequences, a few proposed
// tokens), for one cache type and head_dim.
//
// Such a unit reads its whole context for a few rows: the reads bound it.  A
// 128-row tensor-core tile would be mostly empty, and its round trips through
// tensor memory take longer than the reads, so here every warp multiplies 16 rows
// by 16 keys at a time in registers, over keys of its own, with its own running
// maximum and sum:
//
//   x = c (Q K^T),  m' = max(m, max x),  P = 2^(x - m'),  l = l 2^(m - m') + sum P,
//   O = O 2^(m - m') + P V
//
// (m moves only when x exceeds it by 8: P <= 2^8.)  The warps of a CTA are joined
// at the segment's end through shared memory.  With more than 16 rows the warps
// form two halves of 16 rows each that read the same keys.
//
// The keys come by asynchronous copies through shared memory.  A lane copies
// exactly the bytes that its own fragments need, so a warp waits for nobody:
// with i = lane / 4, q = lane % 4, a lane has of K the pieces q, q + 4, ... (16
// bytes each) of keys i and i + 8, and of V, of keys 2q, 2q + 1, 8 + 2q and 9 + 2q, the
// pieces i, i + 8, ...  The products' inner and outer orders follow that: any
// order of a score's products serves as long as Q has the same, and V's columns
// are put back in order at the join.  Copies of keys past the context's end
// are filled with zeros, so nothing is read that no sequence owns.
#pragma once

#include "attn_codes.cuh"

namespace ssd {
namespace {

constexpr int kFewWarps = 8;
constexpr float kFewRescale = 8.f;   // log2

template <int kType, int kDim>
struct FewCfg {
    static constexpr bool kQuant = kType != SSD_KV_BF16;
    static constexpr int kRowBytes = kQuant ? kDim : 2 * kDim;
    static constexpr int kLaneBytes = kRowBytes / 2;          // of 16 keys, a lane's 1 / 32
    static constexpr int kSlot = 32 * kLaneBytes + (kQuant ? 64 : 0);   // K or V of 16 keys, with scales
    static constexpr int kSlots = 24 * 1024 / kSlot;
    static constexpr int kRing = kSlots * kSlot;              // bytes of a warp
    // a lane's copies: pieces of kPiece bytes
    static constexpr int kKPieces = kLaneBytes / 16;          // 16 bytes each
    static constexpr int kVPiece = kRowBytes >= 128 ? 16 : 8;
    static constexpr int kVPieces = kRowBytes / 8 / kVPiece;  // of each of four keys
    static constexpr int kOOff = kFewWarps * kRing;
    static constexpr int kOBytes = kFewWarps * 16 * kDim * 4;
    static constexpr int kMlOff = kOOff;                      // the join works in the ring's place
    static constexpr int kBytes = kOOff + kFewWarps * 16 * 8 + 128;
};

// Adds to kN columns from d of a row's sums the infinities and NaN that were
// taken out of V: those of the keys in [lo, hi) of groups [ga, gb) that some row
// does not see all of.
template <int kDim, int kN>
__device__ __noinline__ void few_add_nonfinite(const AttnParams &p, const AttnUnit &e, int h, int ga,
                                               int gb, int hi, int lo, int d, float *acc)
{
    for (int gi = ga; gi < gb; ++gi) {
        if (!attn_partial(e, p.window, gi * 16, 16, 0, e.tokens - 1))
            continue;
        for (int j = max(gi * 16, max(lo, 0)); j < min(gi * 16 + 16, hi); ++j) {
            const int64_t page = kv_page_of(p.c, e.seq, j);
            if (page < 0)
                continue;
            const __nv_bfloat16 *v =
                static_cast<const __nv_bfloat16 *>(p.c.v) + kv_row(p.c, page, h, j) * kDim + d;
            for (int k = 0; k < kN; ++k) {
                const float x = __bfloat162float(v[k]);
                if (!(fabsf(x) <= 3.4e38f))
                    acc[k] += x;
            }
        }
    }
}

// The 16-key groups of a segment that a warp works on: those that some row sees,
// every n-th from its own.
struct FewGroups {
    int next, last, step;

    __device__ __forceinline__ void begin(const AttnWalk &w, int window, int lane_group, int groups)
    {
        const int keys = max(w.e.pos0 + w.e.tokens, 0);
        const int first = window > 0 ? max(w.e.pos0 - window + 1, 0) / 16 : 0;
        next = max((w.e.tile0 + w.ta) * (kTileKeys / 16), first) + lane_group;
        last = min((w.e.tile0 + w.tb) * (kTileKeys / 16), (keys + 15) / 16);
        step = groups;
    }
};

template <int kType, int kDim>
__global__ void __launch_bounds__(kFewWarps * 32, 1) attn_few_kernel(const __grid_constant__ AttnParams p)
{
    using C = FewCfg<kType, kDim>;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, i = lane >> 2, q = lane & 3;
    const AttnLine &line = p.line[1];
    const KvView &c = p.c;
    const int g = p.group;
    float *sO = reinterpret_cast<float *>(smem);
    float2 *sMl = reinterpret_cast<float2 *>(smem + C::kMlOff);
    const uint32_t ring = ptx::smem_u32(smem) + warp * C::kRing;
    pdl_launch_dependents();
    // the plan; behind the tiles' kernel, whose CTAs let this one start only after
    // they have seen the plan, nothing more is needed before the end
    if (!p.few_behind_tiles)
        pdl_wait();

    for (AttnWalk w(line, c.heads); w.more(); w.next()) {
        const AttnUnit &e = w.e;
        const int rows = e.tokens * g;
        const bool two = rows > 16;
        const int half = two ? warp / (kFewWarps / 2) : 0;
        FewGroups load;
        load.begin(w, p.window, two ? warp % (kFewWarps / 2) : warp, two ? kFewWarps / 2 : kFewWarps);
        FewGroups work = load;
        // ---- copies of a group's K or V into a slot ----
        int ahead = 32, my_page = 0;             // lane l has the page of the l-th of 32 groups
        int64_t page = 0;
        auto find_page = [&] {
            if (ahead == 32) {
                ahead = 0;
                const int n = load.next + lane * load.step;
                my_page = -1;
                if (n < load.last && n * 16 < e.kv_len)
                    my_page = static_cast<int>(kv_page_of(c, e.seq, n * 16));
            }
            page = __shfl_sync(0xffffffffu, my_page, ahead++);
        };
        auto copy = [&](int slot, int kv) {
            if (load.next < load.last) {
                if (kv == 0)
                    find_page();
                const int j0 = load.next * 16, left = page < 0 ? 0 : e.kv_len - j0;
                const int64_t row = kv_row(c, page < 0 ? 0 : page, w.h, j0);
                const uint8_t *src = static_cast<const uint8_t *>(kv ? c.v : c.k) + row * C::kRowBytes;
                const uint32_t dst = ring + slot * C::kSlot;
                if (kv == 0) {
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int k = 0; k < C::kKPieces / 2; ++k)
                            ptx::cp_async<16>(dst + ((n * (C::kKPieces / 2) + k) * 32 + lane) * 16,
                                              src + (n * 8 + i) * C::kRowBytes + (k * 4 + q) * 16,
                                              n * 8 + i < left);
                } else {
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const int key = q * 2 + (n & 1) + (n >> 1) * 8;
#pragma unroll
                        for (int k = 0; k < C::kVPieces; ++k)
                            ptx::cp_async<C::kVPiece>(
                                dst + ((n * C::kVPieces + k) * 32 + lane) * C::kVPiece,
                                src + key * C::kRowBytes + (k * 8 + i) * C::kVPiece, key < left);
                    }
                }
                if constexpr (C::kQuant) {
                    if (lane < 4)
                        ptx::cp_async<16>(dst + 32 * C::kLaneBytes + lane * 16,
                                          (kv ? c.v_scale : c.k_scale) + row + lane * 4, left > 0);
                }
                if (kv)
                    load.next += load.step;
            }
            ptx::cp_async_commit();
        };
        int put = 0, got = 0;                    // slots
        uint32_t odd = 0;
        auto copy_next = [&] {
            copy(put, odd);
            odd ^= 1;
            put = put + 1 == C::kSlots ? 0 : put + 1;
        };
#pragma unroll 1
        for (int k = 0; k < C::kSlots - 1; ++k)
            copy_next();

        // ---- this lane's rows: Q, and the keys that they see ----
        int lo[2], hi[2];
        uint32_t qa[kDim / 16][4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = half * 16 + i + r * 8, tok = row / g;
            const int pos = e.pos0 + min(tok, e.tokens - 1);
            hi[r] = pos + 1;
            lo[r] = p.window > 0 ? pos - p.window + 1 : INT32_MIN / 2;
            const uint4 *src = reinterpret_cast<const uint4 *>(
                p.q + (e.row0 + tok) * p.q_stride + static_cast<int64_t>(w.h * g + row % g) * kDim);
#pragma unroll
            for (int k = 0; k < kDim / 32; ++k) {
                // (piece of eight elements, in the order of K's pieces)
                const int at = C::kQuant ? (k >> 1) * 8 + q * 2 + (k & 1) : k * 4 + q;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (row < rows)
                    v = src[at];
                const uint32_t flip = p.negate ? 0x80008000u : 0u;
                qa[2 * k][r] = v.x ^ flip;
                qa[2 * k][2 + r] = v.y ^ flip;
                qa[2 * k + 1][r] = v.z ^ flip;
                qa[2 * k + 1][2 + r] = v.w ^ flip;
            }
        }
        float o[kDim / 8][4];
#pragma unroll
        for (int s = 0; s < kDim / 8; ++s)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                o[s][k] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        bool nonfinite = false;

        for (; work.next < work.last; work.next += work.step) {
            const int j0 = work.next * 16;
            const bool hides = attn_partial(e, p.window, j0, 16, 0, e.tokens - 1);
            // ---- scores ----
            ptx::cp_async_wait<C::kSlots - 2>();
            __syncwarp();                        // the other lanes' copies of the scales
            const uint8_t *slot = smem + warp * C::kRing + got * C::kSlot;
            got = got + 1 == C::kSlots ? 0 : got + 1;
            copy_next();
            float x[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    x[n][k] = 0.f;
#pragma unroll
                for (int k = 0; k < C::kKPieces / 2; ++k) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(
                        slot + ((n * (C::kKPieces / 2) + k) * 32 + lane) * 16);
                    if constexpr (C::kQuant) {
                        const uint32_t v4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int s = 0; s < 4; ++s) {
                            uint32_t b[2];
                            widen4<kType>(v4[s], b);
                            ptx::mma_16816(x[n], qa[k * 4 + s], b[0], b[1]);
                        }
                    } else {
                        ptx::mma_16816(x[n], qa[2 * k], v.x, v.y);
                        ptx::mma_16816(x[n], qa[2 * k + 1], v.z, v.w);
                    }
                }
            }
            if constexpr (C::kQuant) {
                const float *sc = reinterpret_cast<const float *>(slot + 32 * C::kLaneBytes);
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float2 f = *reinterpret_cast<const float2 *>(sc + n * 8 + q * 2);
                    x[n][0] *= f.x;
                    x[n][1] *= f.y;
                    x[n][2] *= f.x;
                    x[n][3] *= f.y;
                }
            }
            if (hides) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int j = j0 + n * 8 + q * 2 + (k & 1);
                        if (j < lo[k >> 1] || j >= hi[k >> 1])
                            x[n][k] = -INFINITY;
                    }
            }
            // ---- probabilities ----
            float mx[2];
            bool up = false;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                mx[r] = fmaxf(fmaxf(x[0][2 * r], x[0][2 * r + 1]), fmaxf(x[1][2 * r], x[1][2 * r + 1])) *
                        p.scale_log2;
                up = up || mx[r] > m[r] + kFewRescale;
            }
            if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float v = mx[r];
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
                    const float mn = fmaxf(m[r], v);
                    const float f = mn == m[r] ? 1.f : ptx::ex2(m[r] - mn);
                    m[r] = mn;
                    l[r] *= f;
#pragma unroll
                    for (int s = 0; s < kDim / 8; ++s) {
                        o[s][2 * r] *= f;
                        o[s][2 * r + 1] *= f;
                    }
                }
            }
            float pr[2][4];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float nm = m[r] == -INFINITY ? 0.f : -m[r];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    pr[n][2 * r] = ptx::ex2(fmaf(x[n][2 * r], p.scale_log2, nm));
                    pr[n][2 * r + 1] = ptx::ex2(fmaf(x[n][2 * r + 1], p.scale_log2, nm));
                    l[r] += pr[n][2 * r] + pr[n][2 * r + 1];
                }
            }
            // ---- P V ----
            ptx::cp_async_wait<C::kSlots - 2>();
            __syncwarp();
            slot = smem + warp * C::kRing + got * C::kSlot;
            got = got + 1 == C::kSlots ? 0 : got + 1;
            copy_next();
            if constexpr (C::kQuant) {
                const float *sc = reinterpret_cast<const float *>(slot + 32 * C::kLaneBytes);
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float2 f = *reinterpret_cast<const float2 *>(sc + n * 8 + q * 2);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        // (a hidden key's scale may be NaN: its weight stays zero)
                        const float t = pr[n][k] * (k & 1 ? f.y : f.x);
                        pr[n][k] = hides && pr[n][k] == 0.f ? 0.f : t;
                    }
                }
            }
            const uint32_t pa[4] = {pack_bf16(pr[0][0], pr[0][1]), pack_bf16(pr[0][2], pr[0][3]),
                                    pack_bf16(pr[1][0], pr[1][1]), pack_bf16(pr[1][2], pr[1][3])};
#pragma unroll
            for (int k = 0; k < C::kVPieces; ++k) {
                constexpr int kWords = C::kVPiece / 4;
                uint32_t v[4][kWords];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const uint8_t *src = slot + ((n * C::kVPieces + k) * 32 + lane) * C::kVPiece;
                    if constexpr (kWords == 4) {
                        const uint4 t = *reinterpret_cast<const uint4 *>(src);
                        v[n][0] = t.x;
                        v[n][1] = t.y;
                        v[n][2] = t.z;
                        v[n][3] = t.w;
                    } else {
                        const uint2 t = *reinterpret_cast<const uint2 *>(src);
                        v[n][0] = t.x;
                        v[n][1] = t.y;
                    }
                }
                if constexpr (C::kQuant) {
#pragma unroll
                    for (int s = 0; s < kWords; ++s) {
                        uint32_t a[2], b[2];
                        widen_columns<kType, 0>(v[0][s], v[1][s], a);
                        widen_columns<kType, 0>(v[2][s], v[3][s], b);
                        ptx::mma_16816(o[s * 4], pa, a[0], b[0]);
                        ptx::mma_16816(o[s * 4 + 1], pa, a[1], b[1]);
                        widen_columns<kType, 2>(v[0][s], v[1][s], a);
                        widen_columns<kType, 2>(v[2][s], v[3][s], b);
                        ptx::mma_16816(o[s * 4 + 2], pa, a[0], b[0]);
                        ptx::mma_16816(o[s * 4 + 3], pa, a[1], b[1]);
                    }
                } else {
                    if (hides) {
                        // infinities and NaN would reach the rows that do not see them
                        // (0 times them): they are added at the end to those that do
#pragma unroll
                        for (int n = 0; n < 4; ++n)
#pragma unroll
                            for (int s = 0; s < 4; ++s) {
                                const bool a = (v[n][s] & 0x7f80u) == 0x7f80u;
                                const bool b = (v[n][s] & 0x7f800000u) == 0x7f800000u;
                                nonfinite = nonfinite || a || b;
                                v[n][s] &= (a ? 0xffff0000u : 0xffffffffu) & (b ? 0xffffu : 0xffffffffu);
                            }
                    }
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        ptx::mma_16816(o[k * 8 + 2 * s], pa, __byte_perm(v[0][s], v[1][s], 0x5410),
                                       __byte_perm(v[2][s], v[3][s], 0x5410));
                        ptx::mma_16816(o[k * 8 + 2 * s + 1], pa, __byte_perm(v[0][s], v[1][s], 0x7632),
                                       __byte_perm(v[2][s], v[3][s], 0x7632));
                    }
                }
            }
        }

        // ---- join the warps, in the ring's place ----
        ptx::cp_async_wait<0>();
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            if (q == 0)
                sMl[warp * 16 + i + r * 8] = make_float2(m[r], l[r]);
        }
        const bool clean = !__syncthreads_or(nonfinite);
        const int warps = two ? kFewWarps / 2 : kFewWarps;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = i + r * 8;
            float top = -INFINITY;
            for (int k = 0; k < warps; ++k)
                top = fmaxf(top, sMl[(half * warps + k) * 16 + row].x);
            const float f = m[r] == -INFINITY ? 0.f : ptx::ex2(m[r] - top);
            // (16-byte pieces XOR the row, so that the rows of a store meet other banks)
            float *dst = sO + (warp * 16 + row) * kDim;
#pragma unroll
            for (int s = 0; s < kDim / 8; s += 4)
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    // columns of product s, n: i = 2q + n
                    const int d = C::kQuant ? (2 * q + n) * (kDim / 8) + s
                                            : (s / 8) * 64 + (2 * q + n) * 8 + s % 8;
                    *reinterpret_cast<float4 *>(dst + (((d >> 2) ^ (row & 7)) << 2)) =
                        make_float4(o[s][2 * r + n] * f, o[s + 1][2 * r + n] * f,
                                    o[s + 2][2 * r + n] * f, o[s + 3][2 * r + n] * f);
                }
        }
        __syncthreads();
        constexpr int kPieces = kDim / 8;        // a thread's eight elements
        for (int x = tid; x < rows * kPieces; x += kFewWarps * 32) {
            const int row = x / kPieces, d = (x % kPieces) * 8, r16 = row & 15;
            const int w0 = two ? (row >> 4) * warps : 0;
            float top = -INFINITY, sum = 0.f;
            for (int k = 0; k < warps; ++k)
                top = fmaxf(top, sMl[(w0 + k) * 16 + r16].x);
            float acc[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                acc[k] = 0.f;
            for (int k = 0; k < warps; ++k) {
                const float2 ml = sMl[(w0 + k) * 16 + r16];
                sum += ml.x == -INFINITY ? ml.y : ptx::ex2(ml.x - top) * ml.y;
                const float *src = sO + ((w0 + k) * 16 + r16) * kDim;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float4 v =
                        *reinterpret_cast<const float4 *>(src + (((d / 4 + n) ^ (r16 & 7)) << 2));
                    acc[4 * n] += v.x;
                    acc[4 * n + 1] += v.y;
                    acc[4 * n + 2] += v.z;
                    acc[4 * n + 3] += v.w;
                }
            }
            const int tok = row / g, pos = e.pos0 + tok;
            if (!clean)
                few_add_nonfinite<kDim, 8>(p, e, w.h, (e.tile0 + w.ta) * (kTileKeys / 16),
                                           (e.tile0 + w.tb) * (kTileKeys / 16), pos + 1,
                                           p.window > 0 ? pos - p.window + 1 : 0, d, acc);
            const int64_t grow = e.row0 + tok;
            const int head = w.h * g + row % g;
            if (w.whole()) {
                const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
                *reinterpret_cast<uint4 *>(p.o + grow * p.o_stride + static_cast<int64_t>(head) * kDim + d) =
                    make_uint4(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv),
                               pack_bf16(acc[4] * inv, acc[5] * inv), pack_bf16(acc[6] * inv, acc[7] * inv));
                if (p.lse && d == 0)
                    p.lse[grow * p.heads + head] =
                        sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
            } else {
                const int64_t prow = attn_slot(blockIdx.x, w.starts()) * kFewRows + row;
                float4 *dst = reinterpret_cast<float4 *>(line.part_o + prow * kDim + d);
                dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
                dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
                if (d == 0)
                    line.part_ml[prow] = make_float2(top, sum);
            }
        }
        __syncthreads();
    }
    // this grid ends after its predecessors, so that the join may rely on them all
    pdl_wait();
}

template <int kType, int kDim>
cudaError_t launch_few_one(const AttnParams &p, cudaStream_t stream)
{
    using C = FewCfg<kType, kDim>;
    static_assert(C::kBytes <= kMaxSmemPerBlock && C::kOBytes <= C::kOOff && C::kSlots >= 4, "shared memory");
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
