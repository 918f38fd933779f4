// The attention kernel, for one cache type and head_dim.
//
// For the query rows of a unit (whole tokens with the query heads of one kv
// head, packed into one or two 128-row tiles, "streams") and its key tiles of
// 128 keys:
//
//   S = Q K^T                       (tcgen05, both operands in shared memory)
//   m' = max(m, max_j S_j),  P = 2^(c S - c m'),  l = l 2^(c m - c m') + sum P
//   O = O 2^(c m - c m') + P V      (tcgen05, P in tensor memory, V in shared memory)
//
// with c = softmax_scale log2(e): one pass over the keys with the running
// maximum and sum of the softmax.  A row keeps an old reference m until its
// probabilities of half a tile add up to more than 2^16, so that O is rescaled a few
// times per row and not per tile; neither the fp32 sums nor the bf16 operand feel
// the factor.  So the probabilities are computed at once with the reference at hand,
// and only then is it known whether it served.
//
// One CTA per SM, 16 warps (8-bit caches: 20).  The two streams share every key tile,
// which halves the reads of K and V per query row, and take turns: while one stream's
// warps exponentiate, the tensor cores run the other's products.  A tile's scores come
// in two halves of 64 keys, so that the first half's probabilities are there before
// the second half's scores are (830 us as a whole, 796 in halves).
//   warps 0-3, 4-7   softmax and output of stream 0 and 1: 64 scores a thread, of one
//                    row or of four; probabilities are rounded once, to bf16, the
//                    operand's type, in the scores' place
//   four warps more  bf16: clean the V tiles that hold rows nobody may see;
//   (8-bit: eight)   8-bit: widen codes to bf16 tiles (exact: 8 bits at most)
//   one              TMA producer: Q, K and V page by page
//   two              tcgen05 issuers of stream 0 and 1
//
// Masks are looked at by warp and half tile: with a mask for the whole tile, four
// sequences of 700 to 1,111 tokens with a window of 1,024 take 73 us, 63 so.
//
// Measured: 2,048 tokens of 32 heads over 32,768 keys of 8 kv heads of 128, bf16:
// 750 us, 1.42 PFLOP/s, 73 % of the burst rate of a plain matrix product; the tensor
// pipes are busy 80 % of the time, at the board's power limit.  The same heads, two
// sequences of 1,024 tokens over 12,001 to 16,383 fp8 keys: 484 us, 0.93 PFLOP/s; there
// the softmax and the widening share the schedulers and shared memory, and the way
// from a code to a product is long (with three tiles for products and three of codes
// instead of four and one: 14 us more).
#pragma once

#include "attn_codes.cuh"
#include "kernels.cuh"

namespace ssd {
namespace {

constexpr int kBlk = kTileKeys * 128;      // 128 rows of 64 bf16: one swizzled block
constexpr uint32_t kTmemCols = 512;
constexpr int kSlots8 = 4;                 // scale tiles in flight (8-bit caches)
constexpr float kRescale = 65536.f;      // a half tile's sum of probabilities that asks for it

template <int kType, int kDim>
struct Cfg {
    static constexpr bool kQuant = kType != SSD_KV_BF16;
    // warps: 8 of softmax, the helpers, producer, two issuers, one idle; registers a
    // thread at launch, and after the split
    static constexpr int kHelpers = kQuant ? 8 : 4;
    static constexpr int kProducer = 8 + kHelpers, kIssuer = kProducer + 1;
    static constexpr int kThreads = (kProducer + 4) * 32;
    static constexpr int kLaunchRegs = kQuant ? 96 : 128;
    static constexpr int kSoftmaxRegs = kQuant ? 152 : 168, kOtherRegs = kQuant ? 56 : 88;
    static_assert(256 * kSoftmaxRegs + (kThreads - 256) * kOtherRegs <= kThreads * kLaunchRegs &&
                  kThreads * kLaunchRegs <= 65536, "registers");
    static constexpr int kBlocks = kDim / 64;
    static constexpr int kTile = kBlocks * kBlk;             // a bf16 tile of 128 rows
    static constexpr int kRaw = kTileKeys * kDim;            // the same in 8-bit codes
    static constexpr int kStages = (kQuant ? 4 : 5) * (128 / kDim) - (kQuant || kDim == 128 ? 0 : 2);
    static constexpr int kRawStages = kQuant ? 128 / kDim : 0;
    // shared memory, from a 1024-byte boundary
    static constexpr int kQOff = 0;
    static constexpr int kKvOff = kQOff + 2 * kTile;
    static constexpr int kRawOff = kKvOff + kStages * kTile;
    static constexpr int kScaleOff = kRawOff + kRawStages * kRaw;
    static constexpr int kOnesOff = kScaleOff + (kQuant ? kSlots8 * 2 * kTileKeys * 4 : 0);
    static constexpr int kBarOff = kOnesOff + (kQuant ? kTileKeys / 2 * 4 : 0);
    static constexpr int kBytes = kBarOff + 512 + 1024;
    // tensor memory: per stream 128 columns of S (P in the first 64) and kDim of O
    static constexpr uint32_t kColO = 256;
};

// Barriers, in 8-byte words from kBarOff.  [2][2]: stream, then half of a key tile.
enum Bar {
    kQFull = 0,
    kQEmpty,
    kSFull,              // [2][2] scores are in tensor memory
    kPFull = kSFull + 4, // [2][2] probabilities are
    kPvDone = kPFull + 4, // [2][2] their product is done
    kOFull = kPvDone + 4, // [2] a segment's last product is
    kFixReq = kOFull + 2,
    kFixDone,
    kDrain,                       // [2]
    kKvFull = kDrain + 2,         // [8]
    kKvEmpty = kKvFull + 8,       // [8]
    kRawFull = kKvEmpty + 8,      // [6]
    kRawEmpty = kRawFull + 6,     // [6]
    kScFull = kRawEmpty + 6,      // [4]
    kScEmpty = kScFull + kSlots8, // [4]
    kNumBars = kScEmpty + kSlots8,
};
static_assert(kNumBars * 8 + 16 <= 512, "barrier space");

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Adds to 32 columns from d of a row's sums the infinities and NaN that were taken
// out of V: those of the keys in [lo, hi) of tiles [ta, tb) that some row of the
// unit does not see all of.
template <int kDim>
__device__ __noinline__ void add_nonfinite(const AttnParams &p, const AttnUnit &e, int h, int ta, int tb,
                                           int hi, int lo, int d, float *acc)
{
    for (int t = ta; t < tb; ++t) {
        const int k0 = (e.tile0 + t) * kTileKeys;
        if (!attn_partial(e, p.window, k0, kTileKeys, 0, e.tokens - 1))
            continue;
        for (int j = max(k0, max(lo, 0)); j < min(k0 + kTileKeys, hi); ++j) {
            const int64_t page = kv_page_of(p.c, e.seq, j);
            if (page < 0)
                continue;
            const __nv_bfloat16 *v =
                static_cast<const __nv_bfloat16 *>(p.c.v) + kv_row(p.c, page, h, j) * kDim + d;
            for (int k = 0; k < 32; ++k) {
                const float x = __bfloat162float(v[k]);
                if (!(fabsf(x) <= 3.4e38f))
                    acc[k] += x;
            }
        }
    }
}

template <int kType, int kDim>
__global__ void __launch_bounds__(Cfg<kType, kDim>::kThreads, 1)
    attn_kernel(const __grid_constant__ AttnMaps maps, const __grid_constant__ AttnParams p)
{
    using C = Cfg<kType, kDim>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sQ = smem + C::kQOff, *sKv = smem + C::kKvOff, *sRaw = smem + C::kRawOff;
    float *sScale = reinterpret_cast<float *>(smem + C::kScaleOff);
    float *sOnes = reinterpret_cast<float *>(smem + C::kOnesOff);   // factors of scores that have theirs
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kBarOff);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kNumBars);
    volatile int *s_abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    // infinities or NaN were taken out of some V tile: from then on the output of every
    // segment looks its masked tiles over for what to add back
    volatile int *s_nonfinite = s_abort + 1;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);     // the same in every lane

    if (tid == 0) {
        ptx::prefetch_tensormap(&maps.Q);
        ptx::prefetch_tensormap(&maps.K);
        ptx::prefetch_tensormap(&maps.V);
        for (int k = 0; k < kNumBars; ++k) {
            const bool many = k == kFixDone || (k >= kRawEmpty && k < kScFull) ||
                              (C::kQuant && k >= kKvFull && k < kKvEmpty);   // the helpers
            const bool warps = k >= kPFull && k < kPvDone;
            // what both issuers release
            const bool both = k == kQEmpty || k == kFixReq || (k >= kKvEmpty && k < kRawFull) || k >= kScEmpty;
            ptx::mbar_init(bars + k, many ? C::kHelpers * 32 : warps ? 4 : both ? 2 : 1);
        }
        ptx::fence_barrier_init();
        *s_abort = 0;
        *s_nonfinite = 0;
    }
    if (C::kQuant && tid < kTileKeys / 2)
        sOnes[tid] = 1.f;
    if (warp == C::kIssuer) {
        ptx::tmem_alloc(tmem_slot, kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    pdl_wait();                                // the plan
    pdl_launch_dependents();                   // (its CTAs start as these end, and wait)
    const int g = p.group, tt = p.tile_tokens;
    bool ok = true;
    auto streams = [&](const AttnUnit &e) { return e.tokens > tt ? 2 : 1; };
    auto partial = [&](const AttnUnit &e, int t, int first, int last) {
        return attn_partial(e, p.window, (e.tile0 + t) * kTileKeys, kTileKeys, first, last);
    };
    // Waits, after which the warp goes on together or leaves its loops together.  (A
    // test answers sooner where the barrier is through already, 56 against 86 cycles;
    // polling with it took more issue slots than it won: 782 against 756 us for 2048
    // tokens over 32,768 keys.)
    auto lazy_wait = [&](int bar, uint32_t parity) {
        ok = ok && ptx::mbar_wait(bars + bar, parity & 1, kWaitTimeoutNs) && !*s_abort;
        ok = __all_sync(0xffffffffu, ok);
        return ok;
    };
    auto wait = [&](int bar, uint32_t parity) {
        if (__all_sync(0xffffffffu, ptx::mbar_test(ptx::smem_u32(bars + bar), parity & 1)))
            return ok;
        return lazy_wait(bar, parity);
    };

    if (warp == C::kProducer) {
        ptx::setmaxnreg_dec<C::kOtherRegs>();
        // ------------------------------------------------------------ producer
        uint32_t it = 0, qit = 0, sit = 0;     // tiles, segments, key tiles so far
        constexpr int kRing = C::kQuant ? C::kRawStages : C::kStages;
        constexpr int kFull = C::kQuant ? kRawFull : kKvFull, kEmpty = C::kQuant ? kRawEmpty : kKvEmpty;
        const int shift = p.c.page_shift;
        const int boxes = shift >= 7 ? 1 : kTileKeys >> shift;    // pages of a tile
        for (AttnWalk w(p.line[0], p.c.heads, blockIdx.x); w.more() && ok; w.next(), ++qit) {
            const int ns = streams(w.e);
            if (qit > 0 && !lazy_wait(kQEmpty, qit - 1))
                break;
            if (lane == 0) {
                ptx::mbar_arrive_expect_tx(bars + kQFull, ns * g * tt * kDim * 2);
                for (int st = 0; st < ns; ++st)
                    for (int b = 0; b < C::kBlocks; ++b)
                        ptx::tma_load_3d(sQ + st * C::kTile + b * kBlk, &maps.Q, bars + kQFull,
                                         b * 64, w.h * g, w.e.row0 + st * tt);
            }
            for (int t = w.ta; t < w.tb && ok; ++t, ++sit) {
                // this lane's page of the tile; beyond the sequence's keys, or with
                // an index out of range, one past the cache: it reads as zeros
                const int j0 = (w.e.tile0 + t) * kTileKeys + (lane << shift);
                int64_t page = p.c.num_pages;
                if (lane < boxes && j0 < w.e.kv_len) {
                    const int64_t got = kv_page_of(p.c, w.e.seq, j0);
                    page = got < 0 ? page : got;
                }
                const int z = static_cast<int>(page * p.c.heads) + w.h;
                const int y = shift > 7 ? j0 & (p.c.page - 1) : 0;
                if constexpr (C::kQuant) {
                    const int slot = sit % kSlots8;
                    if (sit >= kSlots8 && !lazy_wait(kScEmpty + slot, sit / kSlots8 - 1))
                        break;
                    // untiled copies (a page's scales may be 64 bytes, less than a tiled
                    // copy's alignment), so zeros are written here
                    const bool there = lane < boxes && page < p.c.num_pages;
                    const uint32_t bytes = min(p.c.page, kTileKeys) * 4;
                    float *dst = sScale + slot * 2 * kTileKeys + (lane << shift);
                    if (lane < boxes && !there) {
                        for (int k = 0; k < static_cast<int>(bytes) / 4; ++k)
                            dst[k] = dst[kTileKeys + k] = 0.f;
                        ptx::fence_proxy_async_smem();
                    }
                    const uint32_t n = __popc(__ballot_sync(0xffffffffu, there));
                    __syncwarp();        // the lanes' zeros, before the arrival that lets them be read
                    if (lane == 0)
                        ptx::mbar_arrive_expect_tx(bars + kScFull + slot, n * 2 * bytes);
                    __syncwarp();
                    if (there) {
                        const int64_t at = static_cast<int64_t>(z) * p.c.page + y;
                        ptx::bulk_load(dst, p.c.k_scale + at, bytes, bars + kScFull + slot);
                        ptx::bulk_load(dst + kTileKeys, p.c.v_scale + at, bytes, bars + kScFull + slot);
                    }
                }
                for (int kv = 0; kv < 2 && ok; ++kv, ++it) {
                    const int s = it % kRing;
                    if (it >= kRing && !lazy_wait(kEmpty + s, it / kRing - 1))
                        break;
                    if (lane == 0)
                        ptx::mbar_arrive_expect_tx(bars + kFull + s, C::kQuant ? C::kRaw : C::kTile);
                    __syncwarp();
                    if (lane < boxes) {
                        const CUtensorMap *m = kv ? &maps.V : &maps.K;
                        if constexpr (C::kQuant) {
                            ptx::tma_load_3d(sRaw + s * C::kRaw + ((lane << shift) * kDim), m,
                                             bars + kFull + s, 0, y, z);
                        } else {
                            for (int b = 0; b < C::kBlocks; ++b)
                                ptx::tma_load_3d(sKv + s * C::kTile + b * kBlk + (lane << shift) * 128,
                                                 m, bars + kFull + s, b * 64, y, z);
                        }
                    }
                }
            }
        }
        if (!ok)
            *s_abort = 1;
        // copies still in flight must land before the CTA exits
        if (qit > 0)
            ptx::mbar_wait(bars + kQFull, (qit - 1) & 1, kWaitTimeoutNs);
        if (!ok && lane == 0)
            ptx::mbar_wait(bars + kQFull, qit & 1, kWaitTimeoutNs);
        for (uint32_t k = it > kRing ? it - kRing : 0; k < it; ++k)
            ptx::mbar_wait(bars + kFull + k % kRing, (k / kRing) & 1, kWaitTimeoutNs);
        if constexpr (C::kQuant)
            for (uint32_t k = sit > kSlots8 ? sit - kSlots8 : 0; k < sit; ++k)
                ptx::mbar_wait(bars + kScFull + k % kSlots8, (k / kSlots8) & 1, kWaitTimeoutNs);
    } else if (warp == C::kIssuer || warp == C::kIssuer + 1) {
        ptx::setmaxnreg_dec<C::kOtherRegs>();
        // ------------------------------------------------------------ MMA issuers
        // One warp per stream.  A key tile goes in halves of 64 keys with scores of
        // their own, so that the tensor cores have one half's products while the
        // other half's scores are exponentiated.  The second issuer goes through
        // the tiles also where it has no rows: what both read is released by both.
        const int st = warp - C::kIssuer;
        constexpr uint32_t id_s = ptx::idesc_bf16_f32(128, kTileKeys / 2, 0, 0);
        constexpr uint32_t id_o = ptx::idesc_bf16_f32(128, kDim, 0, 1);
        const uint64_t desc_q = ptx::sdesc_sw128(ptx::smem_u32(sQ + st * C::kTile), 16, 1024);
        const uint64_t desc_k = ptx::sdesc_sw128(ptx::smem_u32(sKv), 16, 1024);
        const uint64_t desc_v = ptx::sdesc_sw128(ptx::smem_u32(sKv), kBlk, 1024);
        const uint32_t col_s = tmem + st * 128, col_o = tmem + C::kColO + st * kDim;
        // the ring's position: tiles come as K0 V0 K1 V1 ...
        int s = 0, slot = 0;
        uint32_t phase = 0, q_phase = 0, f_phase = 0, p_phase = 0;
        auto advance = [&] {
            if (++s == C::kStages) {
                s = 0;
                phase ^= 1;
            }
        };
        auto scores = [&](int stage, int half) {
            const uint64_t b = ptx::sdesc_add(desc_k, stage * C::kTile + half * (kBlk / 2));
#pragma unroll
            for (int k = 0; k < kDim / 16; ++k)
                ptx::elect_mma_ss(col_s + half * 64, ptx::sdesc_add(desc_q, (k / 4) * kBlk + (k % 4) * 32),
                                  ptx::sdesc_add(b, (k / 4) * kBlk + (k % 4) * 32), id_s, k != 0);
            ptx::elect_commit(bars + kSFull + st * 2 + half);
        };
        for (AttnWalk w(p.line[0], p.c.heads, blockIdx.x); w.more() && ok; w.next()) {
            const bool mine = __shfl_sync(0xffffffffu, static_cast<int>(streams(w.e) > st), 0) != 0;
            const int n = __shfl_sync(0xffffffffu, w.tb - w.ta, 0);
            if (!wait(kQFull, q_phase) || !wait(kKvFull + s, phase))
                break;
            q_phase ^= 1;
            ptx::tc_fence_after_sync();
            if (mine) {
                scores(s, 0);
                scores(s, 1);
            }
            ptx::elect_commit(bars + kKvEmpty + s);
            if (n == 1)
                ptx::elect_commit(bars + kQEmpty);
            advance();
            for (int t = 0; t < n; ++t) {
                const int vs = s;               // this tile's V, then the next one's K
                if (!wait(kKvFull + vs, phase))
                    break;
                advance();
                const int ks = s;
                const bool more = t + 1 < n;
                if constexpr (!C::kQuant) {
                    if (partial(w.e, w.ta + t, 0, w.e.tokens - 1)) {
                        // (both ask, so that neither can be two answers behind)
                        ptx::elect_arrive(bars + kFixReq);
                        if (!wait(kFixDone, f_phase))
                            break;
                        f_phase ^= 1;
                    }
                }
                if (more) {
                    if (!wait(kKvFull + ks, phase))
                        break;
                    advance();
                }
                if (mine) {
#pragma unroll 1
                    for (int half = 0; half < 2 && ok; ++half) {
                        // P V, then the next tile's scores in P's place
                        wait(kPFull + st * 2 + half, p_phase);
                        ptx::tc_fence_after_sync();
                        const uint64_t b = ptx::sdesc_add(desc_v, vs * C::kTile + half * (kBlk / 2));
#pragma unroll
                        for (int k = 0; k < kTileKeys / 32; ++k)
                            ptx::elect_mma_ts(col_o, col_s + half * 64 + k * 8, ptx::sdesc_add(b, k * 2048),
                                              id_o, t + half + k != 0);
                        ptx::elect_commit(bars + kPvDone + st * 2 + half);
                        if (more)
                            scores(ks, half);
                    }
                    if (!ok)
                        break;
                    p_phase ^= 1;
                    if (!more)
                        ptx::elect_commit(bars + kOFull + st);
                }
                if constexpr (C::kQuant) {      // the stream has read the scales
                    ptx::elect_arrive(bars + kScEmpty + slot);
                    slot = slot + 1 == kSlots8 ? 0 : slot + 1;
                }
                ptx::elect_commit(bars + kKvEmpty + vs);
                if (more)
                    ptx::elect_commit(bars + kKvEmpty + ks);
                if (t + 2 == n)
                    ptx::elect_commit(bars + kQEmpty);
            }
        }
        if (!ok)
            *s_abort = 1;
        // every MMA issued must finish before tensor memory is released
        ptx::elect_commit(bars + kDrain + st);
        ptx::mbar_wait(bars + kDrain + st, 0, kWaitTimeoutNs);
    } else if (warp == C::kIssuer + 2) {
        ptx::setmaxnreg_dec<C::kOtherRegs>();
    } else if (warp >= 8) {
        ptx::setmaxnreg_dec<C::kOtherRegs>();
        const int ht = tid - 256;
        if constexpr (!C::kQuant) {
            // -------------------------------------------------------- V cleaner
            // A key tile that some row may not see all of: rows past the last
            // key (whatever the page holds there) become zeros, and so do
            // infinities and NaN, whose product with a probability of zero
            // would reach rows that do not see them; the output adds them
            // back for the rows that do.
            uint32_t it = 0, fit = 0;
            for (AttnWalk w(p.line[0], p.c.heads, blockIdx.x); w.more() && ok; w.next()) {
                for (int t = w.ta; t < w.tb && ok; ++t, it += 2) {
                    if (!partial(w.e, t, 0, w.e.tokens - 1))
                        continue;
                    if (!lazy_wait(kFixReq, fit++))
                        break;
                    uint8_t *v = sKv + ((it + 1) % C::kStages) * C::kTile;
                    const int keys = w.e.kv_len - (w.e.tile0 + t) * kTileKeys;
                    if (keys < kTileKeys) {
#pragma unroll 1
                        for (int i = ht; i < C::kTile / 16; i += 128)
                            if (((i >> 3) & (kTileKeys - 1)) >= keys)
                                *reinterpret_cast<uint4 *>(v + i * 16) = make_uint4(0, 0, 0, 0);
                    }
                    // (an exponent of ones carries into the sign's place)
                    bool found = false;
                    constexpr int kAtOnce = 8;
                    static_assert(C::kTile / 16 % (128 * kAtOnce) == 0, "a thread's pieces");
#pragma unroll 1
                    for (int i = ht; i < C::kTile / 16; i += 128 * kAtOnce) {
                        uint32_t any = 0;
#pragma unroll
                        for (int k = 0; k < kAtOnce; ++k) {
                            const uint4 x = *reinterpret_cast<const uint4 *>(v + (i + k * 128) * 16);
                            any |= ((x.x & 0x7fff7fffu) + 0x00800080u) | ((x.y & 0x7fff7fffu) + 0x00800080u) |
                                   ((x.z & 0x7fff7fffu) + 0x00800080u) | ((x.w & 0x7fff7fffu) + 0x00800080u);
                        }
                        if (!(any & 0x80008000u))
                            continue;
                        found = true;
#pragma unroll 1
                        for (int k = 0; k < kAtOnce * 4; ++k) {
                            uint32_t *at = reinterpret_cast<uint32_t *>(v + (i + k / 4 * 128) * 16) + k % 4;
                            uint32_t x = *at;
                            if ((x & 0x7f80u) == 0x7f80u)
                                x &= 0xffff0000u;
                            if ((x & 0x7f800000u) == 0x7f800000u)
                                x &= 0xffffu;
                            *at = x;
                        }
                    }
                    if (found)
                        *s_nonfinite = 1;
                    ptx::fence_proxy_async_smem();
                    ptx::mbar_arrive(bars + kFixDone);
                }
            }
        } else {
            // -------------------------------------------------------- converter
            // a thread has one 16-code piece of every kRows-th row: rows alike mod 8, so
            // that its places in the swizzled tile are the same distance apart
            constexpr int kUnits = kDim / 16, kRows = C::kHelpers * 32 / kUnits;
            static_assert(kRows % 8 == 0 && kTileKeys % kRows == 0, "rows of a thread");
            const int row0 = ht / kUnits, c = ht % kUnits;
            const int f = (c >> 2) & 1, c16 = (c & 3) * 2;
            const uint32_t from = row0 * kDim + c * 16;
            // pieces of the second block write their halves in the other order: eight
            // lanes then meet all eight 16-byte banks
            const uint32_t line = (c >> 2) * kBlk + row0 * 128;
            const uint32_t to0 = line + (((c16 + f) ^ (row0 & 7)) << 4);
            const uint32_t to1 = line + (((c16 + 1 - f) ^ (row0 & 7)) << 4);
            uint32_t it = 0, sit = 0;
            for (AttnWalk w(p.line[0], p.c.heads, blockIdx.x); w.more() && ok; w.next())
                for (int t = w.ta; t < w.tb && ok; ++t)
                    for (int kv = 0; kv < 2 && ok; ++kv, ++it) {
                        const int rs = it % C::kRawStages, s = it % C::kStages;
                        if (!wait(kRawFull + rs, it / C::kRawStages))
                            break;
                        if (it >= C::kStages && !wait(kKvEmpty + s, it / C::kStages - 1))
                            break;
                        const int keys = w.e.kv_len - (w.e.tile0 + t) * kTileKeys;
                        float *scale = sScale + (sit % kSlots8) * 2 * kTileKeys;
                        if (kv == 0 && !wait(kScFull + sit % kSlots8, sit / kSlots8))
                            break;
                        sit += kv;
                        const uint8_t *src = sRaw + rs * C::kRaw + from;
                        uint8_t *dst = sKv + s * C::kTile;
                        uint4 x[kTileKeys / kRows];
#pragma unroll
                        for (int k = 0; k < kTileKeys / kRows; ++k)
                            x[k] = *reinterpret_cast<const uint4 *>(src + k * kRows * kDim);
                        ptx::mbar_arrive(bars + kRawEmpty + rs);
                        if (keys < kTileKeys) {
#pragma unroll
                            for (int k = 0; k < kTileKeys / kRows; ++k)
                                if (row0 + k * kRows >= keys)
                                    x[k] = make_uint4(0, 0, 0, 0);
                        }
#pragma unroll
                        for (int k = 0; k < kTileKeys / kRows; ++k) {
                            uint32_t o[8];
                            widen4<kType>(x[k].x, o);
                            widen4<kType>(x[k].y, o + 2);
                            widen4<kType>(x[k].z, o + 4);
                            widen4<kType>(x[k].w, o + 6);
                            *reinterpret_cast<uint4 *>(dst + to0 + k * kRows * 128) =
                                f ? make_uint4(o[4], o[5], o[6], o[7]) : make_uint4(o[0], o[1], o[2], o[3]);
                            *reinterpret_cast<uint4 *>(dst + to1 + k * kRows * 128) =
                                f ? make_uint4(o[0], o[1], o[2], o[3]) : make_uint4(o[4], o[5], o[6], o[7]);
                        }
                        if (kv == 0 && c == 0) {
                            // the rows' scales: K's become the scores' factors (softmax_scale
                            // log2(e) among them); a row that is not finite gets finite ones
                            // and a NaN among its codes, so that scores hidden from a query
                            // stay hidden, and one past the last key any
                            const float c2 = p.negate ? -p.scale_log2 : p.scale_log2;
#pragma unroll
                            for (int k = 0; k < kTileKeys / kRows; ++k) {
                                const int row = row0 + k * kRows;
                                const float ks = scale[row] * c2, vs = scale[kTileKeys + row];
                                const bool bad = !(fabsf(ks) <= 3.4e38f && fabsf(vs) <= 3.4e38f);
                                scale[row] = bad || row >= keys ? c2 : ks;
                                if (bad || row >= keys) {
                                    scale[kTileKeys + row] = 0.f;
                                    if (row < keys)
                                        *reinterpret_cast<uint32_t *>(dst + to0 + k * kRows * 128) = 0x7fff7fffu;
                                }
                            }
                        }
                        ptx::fence_proxy_async_smem();
                        ptx::mbar_arrive(bars + kKvFull + s);
                    }
        }
    } else {
        ptx::setmaxnreg_inc<C::kSoftmaxRegs>();
        // ------------------------------------------------------------ softmax
        // bf16: a thread has all 64 scores of its row.  8-bit caches: scores come in the
        // fragments of a matrix product, with i = lane / 4, q = lane % 4, of rows i, i + 8,
        // i + 16 and i + 24 of the warp the columns 2q and 2q + 1 of every eight, so that
        // a thread needs a quarter of the keys' scales.  (A row's thread needs them all:
        // their 16-byte reads then take more of shared memory's time than the codes,
        // 542 us instead of 484 for the chunks above.  Without scales rows are faster,
        // 50.3 instead of 53.4 us for the windows.)
        constexpr int kR = C::kQuant ? 4 : 1;      // a thread's rows
        constexpr int kPairs = 32 / kR;            // pairs of a row's scores
        const int st = warp >> 2, row = tid & 127, fi = lane >> 2, fq = kR == 4 ? lane & 3 : 0;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t colS = tmem + st * 128 + lanes, colO = tmem + C::kColO + st * kDim + lanes;
        int row_tok[kR];
#pragma unroll
        for (int j = 0; j < kR; ++j)
            row_tok[j] = (kR == 4 ? (warp & 3) * 32 + j * 8 + fi : row) / g;
        const int warp_tok0 = (warp & 3) * 32 / g, warp_tok1 = ((warp & 3) * 32 + 31) / g;
        // of the rows' values, the one of row `lane`
        auto of_row = [&](const float (&v)[kR]) {
            float r = v[0];
            if constexpr (kR == 4) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float x = __shfl_sync(0xffffffffu, v[j], (lane & 7) * 4);
                    r = lane >> 3 == j ? x : r;
                }
            }
            return r;
        };
        const float c2 = p.scale_log2;
        uint32_t it = 0, sit = 0, oit = 0;
        for (AttnWalk w(p.line[0], p.c.heads, blockIdx.x); w.more() && ok; w.next()) {
            if (streams(w.e) <= st) {
                sit += w.tb - w.ta;
                continue;
            }
            const int tok0 = st * tt;
            const int ntok = min(tt, w.e.tokens - tok0);        // tokens of this stream
            // of the warp's rows: first and last position, or none
            const int pos0 = w.e.pos0 + tok0 + warp_tok0;
            const int pos1 = warp_tok0 < ntok ? w.e.pos0 + tok0 + min(warp_tok1, ntok - 1) : INT32_MIN / 2;
            const int back = p.window > 0 ? p.window : INT32_MAX / 2;
            // reference, times c (a row that is none has one, and asks for no other)
            float m[kR], l[kR];
#pragma unroll
            for (int j = 0; j < kR; ++j) {
                m[j] = row_tok[j] < ntok ? -INFINITY : 0.f;
                l[j] = 0.f;
            }
            for (int t = w.ta; t < w.tb && ok; ++t, ++it, ++sit) {
                // (the converter has seen the scales land)
                const float *sc = sScale + (sit % kSlots8) * 2 * kTileKeys + 2 * fq;
#pragma unroll 1
                for (int half = 0; half < 2; ++half, sc += 64) {
                    const uint32_t col = colS + half * 64;
                    const int k0 = (w.e.tile0 + t) * kTileKeys + half * 64;
                    // by warp and half: whether a row does not see all of the keys, and
                    // whether any row sees any
                    const bool hides = k0 + 63 > pos0 || k0 <= pos1 - back;
                    const bool some = k0 <= pos1 && k0 + 63 > pos0 - back;
                    if (!wait(kSFull + st * 2 + half, it))
                        break;
                    ptx::tc_fence_after_sync();
                    // a row's halves, or [rows i, i + 8 | i + 16, i + 24]
                    uint32_t s[2][32], pk[2][16];
                    constexpr int kAcc = kR == 4 ? 4 : 2;
                    uint64_t acc[kAcc];
#pragma unroll
                    for (int j = 0; j < kAcc; ++j)
                        acc[j] = ptx::pack2(0.f, 0.f);
                    if (!some) {
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            pk[0][k] = pk[1][k] = 0;
                    }
#pragma unroll 1
                    for (int pass = 0; some; ++pass) {
                        // ---- 64 scores: sign, hidden keys ----
                        if constexpr (kR == 4) {
                            ptx::tmem_ld_16x64(col, s[0]);
                            ptx::tmem_ld_16x64(col + (16u << 16), s[1]);
                        } else {
                            ptx::tmem_ld32_nowait(col, s[0]);
                            ptx::tmem_ld32_nowait(col + 32, s[1]);
                        }
                        ptx::tmem_wait_ld();
                        // element e of pair k of row j, and its first column
                        auto score = [&](int j, int k, int e) -> uint32_t & {
                            if constexpr (kR == 4)
                                return s[j / 2][k * 4 + j % 2 * 2 + e];
                            else
                                return s[k / 16][k % 16 * 2 + e];
                        };
                        constexpr int kStep = kR == 4 ? 8 : 2;
                        if (!C::kQuant && p.negate) {
#pragma unroll
                            for (int k = 0; k < 32; ++k) {
                                s[0][k] ^= 0x80000000u;
                                s[1][k] ^= 0x80000000u;
                            }
                        }
                        const uint64_t c22 = ptx::pack2(c2, c2);
                        const float *fs = hides ? sOnes + 2 * fq : sc;
                        auto pair = [&](int j, int k) {
                            return ptx::pack2(__uint_as_float(score(j, k, 0)), __uint_as_float(score(j, k, 1)));
                        };
                        if (hides) {
                            if constexpr (C::kQuant) {
                                // to log2 units first: a key's factor may be zero (its page is out
                                // of range) or have any sign, and hidden it is -infinity
#pragma unroll
                                for (int k = 0; k < kPairs; ++k) {
                                    const uint64_t f = *reinterpret_cast<const uint64_t *>(sc + k * 8);
#pragma unroll
                                    for (int j = 0; j < kR; ++j) {
                                        float e0, e1;
                                        ptx::unpack2(ptx::mul2(pair(j, k), f), e0, e1);
                                        score(j, k, 0) = __float_as_uint(e0);
                                        score(j, k, 1) = __float_as_uint(e1);
                                    }
                                }
                            }
                            // (a bit per key: the compiler moves eight to predicates at a time)
                            auto below = [](int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1; };
#pragma unroll
                            for (int j = 0; j < kR; ++j) {
                                const int pos = w.e.pos0 + tok0 + min(row_tok[j], ntok - 1);
                                const int hi = pos + 1 - k0 - 2 * fq;
                                const int lo = p.window > 0 ? hi - p.window : INT32_MIN / 2;
                                const uint32_t v0 = below(hi) & ~below(lo);
                                const uint32_t v1 = below(hi - 32) & ~below(lo - 32);
#pragma unroll
                                for (int k = 0; k < kPairs; ++k)
#pragma unroll
                                    for (int e = 0; e < 2; ++e) {
                                        const int at = k * kStep + e;
                                        uint32_t &x = score(j, k, e);
                                        x = (at < 32 ? v0 : v1) >> (at & 31) & 1 ? x : 0xff800000u;
                                    }
                            }
                        }
                        auto factors = [&](int k) -> uint64_t {    // of pair k, to log2 units
                            if constexpr (C::kQuant)
                                return *reinterpret_cast<const uint64_t *>(fs + k * 8);
                            else
                                return c22;
                        };
                        auto maxima = [&](float (&x)[kR]) {
                            float x2[kAcc];
#pragma unroll
                            for (int j = 0; j < kAcc; ++j)
                                x2[j] = -INFINITY;
#pragma unroll
                            for (int k = 0; k < kPairs; ++k) {
                                const uint64_t f = factors(k);
#pragma unroll
                                for (int j = 0; j < kR; ++j) {
                                    float e0, e1, &to = x2[kR == 4 ? j : k & 1];
                                    ptx::unpack2(ptx::mul2(pair(j, k), f), e0, e1);
                                    to = max3(to, e0, e1);
                                }
                            }
#pragma unroll
                            for (int j = 0; j < kR; ++j) {
                                x[j] = kR == 4 ? x2[j] : fmaxf(x2[0], x2[1]);
                                if constexpr (kR == 4) {
                                    x[j] = fmaxf(x[j], __shfl_xor_sync(0xffffffffu, x[j], 1));
                                    x[j] = fmaxf(x[j], __shfl_xor_sync(0xffffffffu, x[j], 2));
                                }
                            }
                        };
                        // rows that have seen no key take the half's maximum as reference
                        // (O and l are zero)
                        float least = m[0];
#pragma unroll
                        for (int j = 1; j < kR; ++j)
                            least = fminf(least, m[j]);
                        if (__any_sync(0xffffffffu, least == -INFINITY)) {
                            float mx[kR];
                            maxima(mx);
#pragma unroll
                            for (int j = 0; j < kR; ++j)
                                m[j] = m[j] == -INFINITY ? mx[j] : m[j];
                        }
                        // ---- probabilities, and their sum ----
                        uint64_t nm[kR];
#pragma unroll
                        for (int j = 0; j < kR; ++j) {
                            const float me = m[j] == -INFINITY ? 0.f : -m[j];
                            nm[j] = ptx::pack2(me, me);
                        }
#pragma unroll
                        for (int j = 0; j < kAcc; ++j)
                            acc[j] = ptx::pack2(0.f, 0.f);
#pragma unroll
                        for (int k = 0; k < kPairs; ++k) {
                            const uint64_t f = factors(k);
#pragma unroll
                            for (int j = 0; j < kR; ++j) {
                                float e0, e1;
                                ptx::unpack2(ptx::fma2(pair(j, k), f, nm[j]), e0, e1);
                                uint64_t x = ptx::pack2(ptx::ex2(e0), ptx::ex2(e1));
                                uint64_t &to = acc[kR == 4 ? j : k & 1];
                                to = ptx::add2(to, x);
                                if constexpr (C::kQuant)
                                    x = ptx::mul2(x, *reinterpret_cast<const uint64_t *>(sc + kTileKeys + k * 8));
                                ptx::unpack2(x, e0, e1);
                                if constexpr (kR == 4)
                                    pk[j / 2][k * 2 + j % 2] = pack_bf16(e0, e1);
                                else
                                    pk[k / 16][k % 16] = pack_bf16(e0, e1);
                            }
                        }
                        if constexpr (kR == 1)
                            acc[0] = ptx::add2(acc[0], acc[1]);
                        float most = 0.f;        // (not a number: asks as well)
#pragma unroll
                        for (int j = 0; j < kR; ++j) {
                            float a0, a1;
                            ptx::unpack2(acc[j], a0, a1);
                            most = row_tok[j] < ntok && !(a0 + a1 <= kRescale) ? INFINITY : most;
                        }
                        if (pass || !__any_sync(0xffffffffu, most > 0.f))
                            break;
                        // rare: scores far above the reference.  Once the product under way is
                        // done, the rows of the warp take new ones, and the half is done again
                        const bool first = !half && t == w.ta;
                        if (!first && !wait(kPvDone + st * 2 + (half ^ 1), half ? it : it - 1))
                            break;
                        ptx::tc_fence_after_sync();
                        float f[kR], mx[kR];
                        maxima(mx);
#pragma unroll
                        for (int j = 0; j < kR; ++j) {
                            const float mn = fmaxf(m[j], mx[j]);
                            f[j] = mn == m[j] ? 1.f : ptx::ex2(m[j] - mn);
                            m[j] = mn;
                            l[j] *= f[j];
                        }
                        const float by = of_row(f);
#pragma unroll 1
                        for (int k = 0; k < (first ? 0 : kDim); k += 16) {
                            float o[16];
                            uint32_t r[16];
                            ptx::tmem_ld16(colO + k, o);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                r[i] = __float_as_uint(o[i] * by);
                            ptx::tmem_st16(colO + k, r);
                        }
                    }
                    // (in the place of scores already read)
                    if constexpr (kR == 4) {
                        ptx::tmem_st_16x32(col, pk[0]);
                        ptx::tmem_st_16x32(col + (16u << 16), pk[1]);
                    } else {
                        ptx::tmem_st16(col, pk[0]);
                        ptx::tmem_st16(col + 16, pk[1]);
                    }
#pragma unroll
                    for (int j = 0; j < kR; ++j) {
                        float a0, a1;
                        ptx::unpack2(acc[j], a0, a1);
                        l[j] += a0 + a1;
                    }
                    ptx::tmem_wait_st();
                    ptx::tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        ptx::mbar_arrive(bars + kPFull + st * 2 + half);
                }
            }
            if (!ok || !wait(kOFull + st, oit++))
                break;
            ptx::tc_fence_after_sync();
            // ---- output: the segment's rows, or their partial sums ----
            const bool nonfinite = !C::kQuant && *s_nonfinite, whole = w.whole();
            if constexpr (kR == 4) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    l[j] += __shfl_xor_sync(0xffffffffu, l[j], 1);
                    l[j] += __shfl_xor_sync(0xffffffffu, l[j], 2);
                }
            }
            // a thread per row from here on
            const float sum = of_row(l), top = of_row(m);
            const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
            const int my_tok = row / g;
            const bool mine = my_tok < ntok;
            const int64_t grow = w.e.row0 + tok0 + my_tok;
            const int head = w.h * g + row % g;
            const int64_t slot = attn_slot(blockIdx.x, w.starts());
            // where this thread stores: of four rows (its own and its neighbours') a
            // sixteen-byte piece each, so that four lanes fill 64 bytes of a row; a
            // partial result lies by four columns, row by row
            __nv_bfloat16 *dst = p.o + grow * p.o_stride + static_cast<int64_t>(head) * kDim;
            __nv_bfloat16 *to[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint64_t at = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(mine ? dst : nullptr),
                                                (lane & ~3) + j);
                to[j] = reinterpret_cast<__nv_bfloat16 *>(at);
            }
            float4 *part = reinterpret_cast<float4 *>(p.line[0].part_o + slot * (2 * kTileRows * kDim)) +
                           st * 128 + row;
#pragma unroll 1
            for (int k = 0; k < kDim; k += 32) {
                uint32_t o[32];
                __syncwarp();
                ptx::tmem_ld32_nowait(colO + k, o);
                ptx::tmem_wait_ld();
                if (nonfinite && mine) {
                    // the cleaned values of the keys that this row sees
                    float v[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        v[i] = __uint_as_float(o[i]);
                    const int pos = w.e.pos0 + tok0 + my_tok;
                    add_nonfinite<kDim>(p, w.e, w.h, w.ta, w.tb, pos + 1,
                                        p.window > 0 ? pos - p.window + 1 : 0, k, v);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        o[i] = __float_as_uint(v[i]);
                }
                __syncwarp();
                if (whole) {
                    uint32_t v[4][4];               // [piece][word], then [row][word]
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        v[i / 4][i % 4] = pack_bf16(__uint_as_float(o[2 * i]) * inv,
                                                    __uint_as_float(o[2 * i + 1]) * inv);
#pragma unroll
                    for (int bit = 1; bit < 4; bit *= 2)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int i = 0; i < 4 && !(j & bit); ++i) {
                                const bool up = lane & bit;
                                const uint32_t got = __shfl_xor_sync(
                                    0xffffffffu, up ? v[j][i] : v[j | bit][i], bit);
                                v[j][i] = up ? got : v[j][i];
                                v[j | bit][i] = up ? v[j | bit][i] : got;
                            }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (to[j])
                            *reinterpret_cast<uint4 *>(to[j] + k + (lane & 3) * 8) =
                                make_uint4(v[j][0], v[j][1], v[j][2], v[j][3]);
                } else if (mine) {
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        part[(k + i) / 4 * (2 * kTileRows)] =
                            make_float4(__uint_as_float(o[i]), __uint_as_float(o[i + 1]),
                                        __uint_as_float(o[i + 2]), __uint_as_float(o[i + 3]));
                }
            }
            if (mine) {
                if (!w.whole())
                    p.line[0].part_ml[slot * (2 * kTileRows) + st * 128 + row] = make_float2(top, sum);
                else if (p.lse)
                    p.lse[grow * p.heads + head] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
            }
            // (the next segment's first product waits for this warp's next P)
            ptx::tc_fence_before_sync();
        }
    }

    if (!ok)
        *s_abort = 1;
    ptx::tc_fence_before_sync();
    __syncthreads();
    if (tid == 0 && *s_abort)
        kv_error(p.c, SSD_DEVERR_TIMEOUT);
    if (warp == C::kIssuer) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem, kTmemCols);
    }
}

template <int kType, int kDim>
cudaError_t launch_one(const AttnParams &p, const AttnMaps &m, cudaStream_t stream)
{
    using C = Cfg<kType, kDim>;
    static_assert(C::kBytes <= kMaxSmemPerBlock, "shared memory");
    static_assert(C::kStages <= 8 && C::kRawStages <= 6, "barriers");
    static SmemOptIn opted;
    const void *fn = reinterpret_cast<const void *>(attn_kernel<kType, kDim>);
    cudaError_t e = ensure_max_smem(fn, opted);
    if (e != cudaSuccess)
        return e;
    // with fewer registers at launch the split inside the kernel would wait forever:
    // such a build is refused
    static const bool regs_ok = [fn] {
        cudaFuncAttributes a;
        return cudaFuncGetAttributes(&a, fn) == cudaSuccess && a.numRegs == C::kLaunchRegs;
    }();
    if (!regs_ok)
        return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kAttnCtas);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_kernel<kType, kDim>, m, p);
}

template <int kType>
cudaError_t launch_type(const AttnParams &p, const AttnMaps &m, cudaStream_t stream)
{
    return p.c.dim == 128 ? launch_one<kType, 128>(p, m, stream) : launch_one<kType, 64>(p, m, stream);
}

}  // namespace
}  // namespace ssd
