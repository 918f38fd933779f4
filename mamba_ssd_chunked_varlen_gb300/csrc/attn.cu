// Attention over the paged cache: the plan of a call, the join of split rows,
// and the C ABI (argument checks, tensor maps, launches).
#include <algorithm>
#include <cmath>
#include <mutex>

#include "attn.cuh"
#include "kernels.cuh"

namespace ssd {
namespace {

// ---------------------------------------------------------------- plan
// Cuts the call into units (AttnUnit), in the order of the rows, lays their key tiles
// on the two lines and finds where every piece begins.  Every CTA makes the units for
// itself and an eighth of the pieces: one CTA for all took 10 us, eight take 6.5.
// Up to 256 sequences, 256 threads: shorter barriers (a call is 1 us shorter).
constexpr int kPlanThreads = 1024, kPlanSmall = 256;
constexpr int kPlanCtas = 8;
constexpr int kPlanBatch = 4096;    // up to so many sequences, their first units stay on chip,
constexpr int kPlanUnits = 1024;    // and so many units of a kind, their first tiles

// Inclusive sums of kN values over the CTA's threads; `total` gets the sums of all.
template <int kN>
__device__ __forceinline__ void block_scan(int64_t (&v)[kN], int64_t (*scratch)[32], int64_t (&total)[kN])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int k = 0; k < kN; ++k)
        v[k] = warp_inclusive_scan(v[k]);
    __syncthreads();
    if (lane == 31) {
#pragma unroll
        for (int k = 0; k < kN; ++k)
            scratch[k][warp] = v[k];
    }
    __syncthreads();
    if (warp < kN)
        scratch[warp][lane] = warp_inclusive_scan(lane < blockDim.x / 32 ? scratch[warp][lane] : 0);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kN; ++k) {
        total[k] = scratch[k][31];
        v[k] += warp ? scratch[k][warp - 1] : 0;
    }
}

__global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(const __grid_constant__ AttnParams p)
{
    __shared__ int64_t scratch[4][32];
    __shared__ int32_t s_units[kPlanBatch];
    __shared__ int64_t s_cum[2][kPlanUnits];
    const KvView &c = p.c;
    const int tid = threadIdx.x;
    const int unit_tokens = 2 * p.tile_tokens;
    int32_t *seq_units = c.batch <= kPlanBatch ? s_units : p.seq_units;
    pdl_wait();                  // (the launch alone goes ahead of its predecessor's end)
    pdl_launch_dependents();
    int64_t units = 0;
    int bad = 0;
    for (int base = 0; base < c.batch; base += blockDim.x) {
        const int b = base + tid;
        int64_t n[1] = {0}, all[1];
        if (b < c.batch) {
            const int32_t start = c.qsl[b], end = c.qsl[b + 1];
            if (end < start || (b == 0 && start != 0) || (b == c.batch - 1 && end != c.total_len))
                bad = 1;
            else
                n[0] = (static_cast<int64_t>(end) - start + unit_tokens - 1) / unit_tokens;
        }
        const int64_t mine = n[0];
        block_scan(n, scratch, all);
        if (b < c.batch)
            seq_units[b] = static_cast<int32_t>(min(units + n[0] - mine, static_cast<int64_t>(INT32_MAX)));
        units += all[0];
    }
    // (a query_start_loc that fails may count any number of units: none is written)
    bad = __syncthreads_or(bad);
    // this CTA's pieces, of both kinds one after the other
    constexpr int kEach = (attn_max_pieces(0) + attn_max_pieces(1) + kPlanCtas - 1) / kPlanCtas;
    static_assert(kEach <= kPlanSmall, "a piece per thread");
    const int my_piece = blockIdx.x * kEach + tid;
    const int my_kind = my_piece < attn_max_pieces(0) ? 0 : 1;
    const int i = my_piece - (my_kind ? attn_max_pieces(0) : 0);
    const bool has_piece = tid < kEach && i < attn_max_pieces(my_kind);
    AttnPiece pc = {};
    int4 split = make_int4(0, 0, 0, 0);
    if (bad) {
        if (has_piece) {
            const_cast<AttnPiece *>(p.line[my_kind].pieces)[i] = pc;
            p.line[my_kind].split[i] = split;
        }
        if (tid == 0)
            kv_error(c, SSD_DEVERR_BAD_QUERY_START_LOC);
        return;
    }
    int64_t tiles[2] = {0, 0}, count[2] = {0, 0};
    for (int64_t base = 0; base < units; base += blockDim.x) {
        const int64_t u = base + tid;
        AttnUnit e = {};
        int kind = 0;
        if (u < units) {
            // the last sequence whose units begin at or before u (the sequences
            // without rows that begin there as well come before it)
            int lo = 0, hi = c.batch - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (seq_units[mid] <= u)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            const int32_t start = c.qsl[lo], rows = c.qsl[lo + 1] - start;
            const int32_t first = static_cast<int32_t>(u - seq_units[lo]) * unit_tokens;
            e.seq = lo;
            e.row0 = start + first;
            e.tokens = min(unit_tokens, rows - first);
            e.kv_len = kv_len_of(c, lo);
            e.pos0 = e.kv_len - rows + first;
            kind = e.tokens * p.group <= kFewRows;
            const int n = kind ? kFewKeys : kTileKeys;
            const int32_t keys = max(e.pos0 + e.tokens, 0);
            e.tile0 = p.window > 0 ? max(e.pos0 - p.window + 1, 0) / n : 0;
            e.tiles = max((keys + n - 1) / n - e.tile0, 1);
        }
        int64_t v[4], all[4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            v[2 * k] = u < units && kind == k ? e.tiles : 0;
            v[2 * k + 1] = u < units && kind == k;
        }
        block_scan(v, scratch, all);
        if (u < units) {
            const int64_t at = count[kind] + (kind ? v[3] : v[1]) - 1;
            const_cast<AttnUnit *>(p.line[kind].units)[at] = e;
            const int64_t before = tiles[kind] + (kind ? v[2] : v[0]) - e.tiles;
            p.line[kind].cum[at] = before;
            if (at < kPlanUnits)
                s_cum[kind][at] = before;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            tiles[k] += all[2 * k];
            count[k] += all[2 * k + 1];
        }
    }
    __syncthreads();
    if (!has_piece)
        return;
    // where the piece begins; and where that is within a pair that the piece before
    // begins, the pair is one for the join
    const AttnLine &line = p.line[my_kind];
    const int64_t n_units = my_kind ? count[1] : count[0];
    const int64_t total = (my_kind ? tiles[1] : tiles[0]) * c.heads;
    const int pieces = attn_pieces(my_kind, total);
    if (i < pieces) {
        const int64_t *cum = n_units <= kPlanUnits ? s_cum[my_kind] : line.cum;
        // piece i begins at floor(total i / pieces)
        const int64_t each = total / pieces;
        const int rest = static_cast<int>(total - each * pieces);
        auto begin = [&](int k) { return each * k + rest * k / pieces; };
        const int64_t pos = begin(i);
        pc.tiles = static_cast<int32_t>(begin(i + 1) - pos);
        int lo = 0, hi = static_cast<int>(n_units) - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (cum[mid] * c.heads <= pos)
                lo = mid;
            else
                hi = mid - 1;
        }
        const int64_t r = pos - cum[lo] * c.heads;
        pc.e = line.units[lo];
        const int n = pc.e.tiles;
        pc.u = lo;
        // (tiles and heads are below 2^23 and 2^16)
        pc.h = r >> 31 ? static_cast<int32_t>(r / n) : static_cast<int32_t>(r) / n;
        pc.ta = static_cast<int32_t>(r - static_cast<int64_t>(pc.h) * n);
        const int64_t first = pos - pc.ta;
        if (pc.ta > 0 && first >= begin(i - 1)) {
            // the last piece that begins before the pair's end
            const float rate = static_cast<float>(pieces) / static_cast<float>(total);
            int last = min(i + static_cast<int>((n - pc.ta) * rate), pieces - 1);
            while (last + 1 < pieces && begin(last + 1) < first + n)
                ++last;
            while (begin(last) >= first + n)
                --last;
            split = make_int4(pc.e.row0, pc.e.tokens + (pc.h << 9), i - 1, last);
        }
    }
    const_cast<AttnPiece *>(line.pieces)[i] = pc;
    line.split[i] = split;
}

// ---------------------------------------------------------------- join
// Rows whose keys were split over several pieces: with M the largest of the
// pieces' references m_i,  o = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i,  the pieces
// summed in a fixed order.  Two CTAs of 16 warps an SM first close up the list of
// split pairs (warps that each looked for their own rows met many or none: 12 us for
// 256 pairs of 15 rows, 7 so); then a warp takes four rows of the tiles' kind or a row
// of few; a row of more than kJoinWide pieces (a decoding sequence alone on the GPU)
// takes a CTA.  Few rows: two dependent reads of L2 bound it; tiles: their bytes (24
// sequences, 4 of them chunks of 64 to 500 tokens: 33 MB, 15 us).
constexpr int kJoinWarps = 16;
constexpr int kJoinCtas = 2 * kAttnCtas;

// A sum v of a piece by its weight w: an infinity stays one (and NaN is NaN) where the
// weight has underflowed, so that what a row sees does not depend on how it was cut.
__device__ __forceinline__ float weighted(float w, float v)
{
    return fabsf(v) == INFINITY ? v : w * v;
}

// Adds up pieces from, from + step, ... <= last of a row: its sums relative to `top`.
template <int kE>
__device__ __forceinline__ void join_pieces(const AttnLine &line, int part_rows, int first, int from,
                                            int last, int step, int row, float &top, float &sum,
                                            float (&acc)[kE])
{
    const int lane = threadIdx.x & 31;
    top = -INFINITY;
    sum = 0.f;
#pragma unroll
    for (int j = 0; j < kE; ++j)
        acc[j] = 0.f;
    for (int base = from; base <= last; base += 32 * step) {
        // a lane per piece
        const int mine = base + lane * step;
        float2 ml = make_float2(-INFINITY, 0.f);
        if (mine <= last)
            ml = line.part_ml[attn_slot(mine, mine == first) * part_rows + row];
        float m = ml.x;
#pragma unroll
        for (int o = 16; o; o >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float nt = fmaxf(top, m), f = top == nt ? 1.f : exp2f(top - nt);
        const float w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - nt);
        // (a row of NaN may have no reference)
        float s = ml.x == -INFINITY ? ml.y : w * ml.y;
#pragma unroll
        for (int o = 16; o; o >>= 1)
            s += __shfl_xor_sync(0xffffffffu, s, o);
        sum = sum * f + s;
        top = nt;
#pragma unroll
        for (int j = 0; j < kE; ++j)
            acc[j] = weighted(f, acc[j]);
        // eight pieces' loads at a time; those past the last are not read, but zeros
        const int n = min(32, (last - base) / step + 1);
        for (int k0 = 0; k0 < n; k0 += 8) {
            float v[8][kE];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int at = base + (k0 + k) * step;
                const float *src = line.part_o +
                                   (attn_slot(at, at == first) * static_cast<int64_t>(part_rows) + row) *
                                       (32 * kE) +
                                   lane * kE;
                if constexpr (kE == 4) {
                    const float4 x =
                        at <= last ? *reinterpret_cast<const float4 *>(src) : make_float4(0.f, 0.f, 0.f, 0.f);
                    v[k][0] = x.x;
                    v[k][1] = x.y;
                    v[k][2] = x.z;
                    v[k][3] = x.w;
                } else {
                    const float2 x = at <= last ? *reinterpret_cast<const float2 *>(src) : make_float2(0.f, 0.f);
                    v[k][0] = x.x;
                    v[k][1] = x.y;
                }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float wk = __shfl_sync(0xffffffffu, w, k0 + k);
#pragma unroll
                for (int j = 0; j < kE; ++j)
                    acc[j] += weighted(wk, v[k][j]);
            }
        }
    }
}

template <int kDim>
__global__ void __launch_bounds__(kJoinWarps * 32, 2)
    attn_join_kernel(const __grid_constant__ AttnParams p)
{
    constexpr int kE = kDim / 32;
    __shared__ float s_ml[kJoinWarps][2], s_acc[kJoinWarps][kDim];
    constexpr int kThreads = kJoinWarps * 32, kFewPairs = attn_max_pieces(1);
    constexpr int kLoads = (kFewPairs + kThreads - 1) / kThreads;
    static_assert(attn_max_pieces(0) <= kThreads && kLoads * kJoinWarps == 64);
    __shared__ int4 s_tiles[attn_max_pieces(0)], s_few[kFewPairs];
    __shared__ int s_counts[kLoads + 1][kJoinWarps];
    __shared__ int s_wide[attn_max_pieces(1) / kJoinWide + 1], s_n;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = p.group;
    pdl_wait();
    auto write = [&](const int4 &e, int x, float top, float sum, const float (&acc)[kE]) {
        const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
        const int64_t row = e.x + x / g;
        const int head = (e.y >> 9) * g + x % g;
        __nv_bfloat16 *dst = p.o + row * p.o_stride + static_cast<int64_t>(head) * kDim + lane * kE;
#pragma unroll
        for (int j = 0; j < kE; j += 2)
            *reinterpret_cast<uint32_t *>(dst + j) = pack_bf16(acc[j] * inv, acc[j + 1] * inv);
        if (p.lse && lane == 0)
            p.lse[row * p.heads + head] =
                sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
    };
    const int me = blockIdx.x + warp * kJoinCtas, warps = kJoinWarps * kJoinCtas;

    // ---- the pairs of both kinds, closed up; those of very many pieces apart ----
    const AttnLine &tl = p.line[0], &fl = p.line[1];
    if (tid == 0)
        s_n = 0;
    int4 found[kLoads + 1];
    uint32_t which[kLoads + 1];
#pragma unroll
    for (int k = 0; k <= kLoads; ++k) {
        const int at = k < kLoads ? k * kThreads + tid : tid;
        found[k] = make_int4(0, 0, 0, 0);
        if (at < attn_max_pieces(k < kLoads))
            found[k] = (k < kLoads ? fl : tl).split[at];
    }
#pragma unroll
    for (int k = 0; k <= kLoads; ++k) {
        which[k] = __ballot_sync(0xffffffffu, found[k].y != 0);
        if (lane == 0)
            s_counts[k][warp] = __popc(which[k]);
    }
    __syncthreads();
    const int c0 = s_counts[0][2 * lane], c1 = s_counts[0][2 * lane + 1];   // (few: 64 counts)
    const int upto = warp_inclusive_scan(c0 + c1);
    const int upto0 = warp_inclusive_scan(lane < kJoinWarps ? s_counts[kLoads][lane] : 0);
    const int n1 = __shfl_sync(0xffffffffu, upto, 31), n0 = __shfl_sync(0xffffffffu, upto0, 31);
#pragma unroll
    for (int k = 0; k <= kLoads; ++k) {
        const int i = k * kJoinWarps + warp;
        int at = k < kLoads ? __shfl_sync(0xffffffffu, upto - c1 - (i & 1 ? 0 : c0), i / 2 & 31)
                            : __shfl_sync(0xffffffffu, upto0, warp) - __popc(which[k]);
        at += __popc(which[k] & ((1u << lane) - 1));
        if (found[k].y != 0) {
            (k < kLoads ? s_few : s_tiles)[at] = found[k];
            if (k < kLoads && found[k].w - found[k].z >= kJoinWide)
                s_wide[atomicAdd(&s_n, 1)] = at;
        }
    }
    __syncthreads();

    // ---- tiles: items of four rows of a pair ----
    constexpr int kQuads = 2 * kTileRows / 4;
    for (int item = me; item < n0 * kQuads; item += warps) {
        const int4 e = s_tiles[item / kQuads];
        const int x0 = item % kQuads * 4, rows = (e.y & 511) * g;
        if (x0 >= rows)
            continue;
        auto part_row = [&](int x) {
            const int tok = x / g, st = tok / p.tile_tokens;
            return st * kTileRows + (tok - st * p.tile_tokens) * g + x % g;
        };
        // lane 4 k + r: eight pieces' references of row r; then four columns of each 32
        const int r = lane & 3, k = lane >> 2, x = min(x0 + r, rows - 1), row = part_row(x);
        float top = -INFINITY, sum = 0.f, acc[kE][4];
#pragma unroll
        for (int j = 0; j < kE; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[j][i] = 0.f;
        for (int base = e.z; base <= e.w; base += 8) {
            float2 ml = make_float2(-INFINITY, 0.f);
            if (base + k <= e.w)
                ml = tl.part_ml[attn_slot(base + k, base + k == e.z) * attn_part_rows(0) + row];
            float m = ml.x;
#pragma unroll
            for (int o = 4; o < 32; o <<= 1)
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float nt = fmaxf(top, m), f = top == nt ? 1.f : exp2f(top - nt);
            const float w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - nt);
            float s = ml.x == -INFINITY ? ml.y : w * ml.y;
#pragma unroll
            for (int o = 4; o < 32; o <<= 1)
                s += __shfl_xor_sync(0xffffffffu, s, o);
            sum = sum * f + s;
            top = nt;
#pragma unroll
            for (int j = 0; j < kE; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[j][i] = weighted(f, acc[j][i]);
            const int n = min(8, e.w - base + 1);
#pragma unroll 2
            for (int i = 0; i < n; ++i) {
                const float wi = __shfl_sync(0xffffffffu, w, 4 * i + r);
                const float4 *src = reinterpret_cast<const float4 *>(tl.part_o) +
                                    attn_slot(base + i, base + i == e.z) *
                                        static_cast<int64_t>(attn_part_rows(0) * kDim / 4) +
                                    k * attn_part_rows(0) + row;
#pragma unroll
                for (int j = 0; j < kE; ++j) {
                    const float4 v = src[j * 8 * attn_part_rows(0)];
                    acc[j][0] += weighted(wi, v.x);
                    acc[j][1] += weighted(wi, v.y);
                    acc[j][2] += weighted(wi, v.z);
                    acc[j][3] += weighted(wi, v.w);
                }
            }
        }
        if (x0 + r < rows) {
            const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
            const int64_t orow = e.x + x / g;
            const int head = (e.y >> 9) * g + x % g;
            __nv_bfloat16 *dst = p.o + orow * p.o_stride + static_cast<int64_t>(head) * kDim + k * 4;
#pragma unroll
            for (int j = 0; j < kE; ++j)
                *reinterpret_cast<uint2 *>(dst + j * 32) = make_uint2(
                    pack_bf16(acc[j][0] * inv, acc[j][1] * inv), pack_bf16(acc[j][2] * inv, acc[j][3] * inv));
            if (p.lse && k == 0)
                p.lse[orow * p.heads + head] =
                    sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
        }
    }

    // ---- few rows: items of a row of a pair ----
    for (int item = me; item < n1 * kFewRows; item += warps) {
        const int row = item / n1;
        const int4 e = s_few[item - row * n1];
        if (row >= (e.y & 511) * g || e.w - e.z >= kJoinWide)
            continue;
        float top, sum, acc[kE];
        join_pieces<kE>(fl, kFewRows, e.z, e.z, e.w, 1, row, top, sum, acc);
        write(e, row, top, sum, acc);
    }
    for (int i = 0; i < s_n; ++i) {
        const int4 e = s_few[s_wide[i]];
        const int rows = (e.y & 511) * g;
        // (the CTAs may hold the list in different orders: a pair's rows go by the pair)
        for (int row = (blockIdx.x + kJoinCtas - e.z % kJoinCtas) % kJoinCtas; row < rows; row += kJoinCtas) {
            float top, sum, acc[kE];
            join_pieces<kE>(fl, kFewRows, e.z, e.z + warp, e.w, kJoinWarps, row, top, sum, acc);
            if (lane == 0) {
                s_ml[warp][0] = top;
                s_ml[warp][1] = sum;
            }
#pragma unroll
            for (int j = 0; j < kE; ++j)
                s_acc[warp][lane * kE + j] = acc[j];
            __syncthreads();
            if (warp == 0) {
                top = -INFINITY;
                for (int w = 0; w < kJoinWarps; ++w)
                    top = fmaxf(top, s_ml[w][0]);
                sum = 0.f;
#pragma unroll
                for (int j = 0; j < kE; ++j)
                    acc[j] = 0.f;
                for (int w = 0; w < kJoinWarps; ++w) {
                    const float m = s_ml[w][0], f = m == -INFINITY ? 0.f : exp2f(m - top);
                    sum += m == -INFINITY ? s_ml[w][1] : f * s_ml[w][1];
#pragma unroll
                    for (int j = 0; j < kE; ++j)
                        acc[j] += weighted(f, s_acc[w][lane * kE + j]);
                }
                write(e, row, top, sum, acc);
            }
            __syncthreads();
        }
    }
}

// ---------------------------------------------------------------- host
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn()
{
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// Three-dimensional tensor map; what lies outside reads as zeros.
bool make_map(CUtensorMap *m, CUtensorMapDataType type, const void *base, uint64_t d0, uint64_t d1,
              uint64_t d2, uint64_t pitch1, uint64_t pitch2, uint32_t b0, uint32_t b1, uint32_t b2,
              CUtensorMapSwizzle swizzle)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn)
        return false;
    const cuuint64_t dims[3] = {d0, d1, d2};
    const cuuint64_t strides[2] = {pitch1, pitch2};
    const cuuint32_t box[3] = {b0, b1, b2};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, type, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool sizes_ok(int64_t total_len, int32_t batch, int32_t nheads, int32_t nheads_kv, int32_t head_dim)
{
    return total_len >= 0 && total_len <= INT32_MAX / 2 && batch >= 0 && batch <= INT32_MAX / 2 &&
           nheads > 0 && nheads_kv > 0 && nheads_kv <= kKvMaxHeads && nheads % nheads_kv == 0 &&
           nheads / nheads_kv <= kTileRows && (head_dim == 64 || head_dim == 128);
}

}  // namespace
}  // namespace ssd

extern "C" {

size_t ssd_attn_varlen_workspace_size(int64_t total_len, int32_t batch, int32_t nheads,
                                      int32_t nheads_kv, int32_t head_dim)
{
    if (!ssd::sizes_ok(total_len, batch, nheads, nheads_kv, head_dim))
        return 0;
    // for the largest group that so many query heads can have (it needs the most units), so
    // that calls of fewer kv heads fit as well
    return ssd::attn_layout(total_len, batch, std::min(nheads, ssd::kTileRows), head_dim).total;
}

ssd_status_t ssd_attn_varlen_fwd(void *o, float *lse, const void *q, const void *k_cache,
                                 const void *v_cache, const float *k_scale, const float *v_scale,
                                 const int32_t *query_start_loc, const int32_t *kv_lens,
                                 const int32_t *block_table, int64_t total_len, int32_t batch,
                                 int32_t nheads, int32_t nheads_kv, int32_t head_dim,
                                 int64_t num_pages, int32_t page_size, int32_t table_width,
                                 int64_t table_stride, int32_t cache_type, int64_t o_stride,
                                 int64_t q_stride, float softmax_scale, int32_t window,
                                 void *workspace, size_t workspace_bytes, uint32_t *errors,
                                 ssd_stream_t stream_)
{
    using namespace ssd;
    AttnParams p = {};
    const ssd_status_t st =
        kv_check(&p.c, k_cache, v_cache, k_scale, v_scale, query_start_loc, kv_lens, block_table,
                 total_len, batch, nheads_kv, head_dim, num_pages, page_size, table_width,
                 table_stride, cache_type, errors);
    if (st != SSD_OK)
        return st;
    const float scale_log2 = std::fabs(softmax_scale) * 1.4426950408889634f;
    if (nheads <= 0 || nheads % nheads_kv != 0 || window < 0 || !std::isfinite(scale_log2))
        return SSD_ERR_INVALID_ARG;
    if (!sizes_ok(total_len, batch, nheads, nheads_kv, head_dim))
        return SSD_ERR_UNSUPPORTED;
    const int64_t row = static_cast<int64_t>(nheads) * head_dim;
    if (!kv_pitch(&o_stride, row) || !kv_pitch(&q_stride, row))
        return SSD_ERR_INVALID_ARG;
    if (total_len == 0)
        return SSD_OK;
    if (batch == 0 || !o || !q || !kv_aligned16(o) || !kv_aligned16(q))
        return SSD_ERR_INVALID_ARG;
    const int group = nheads / nheads_kv;
    const AttnLayout L = attn_layout(total_len, batch, group, head_dim);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || workspace_bytes < L.total)
        return SSD_ERR_WORKSPACE;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.o = static_cast<__nv_bfloat16 *>(o);
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.lse = lse;
    p.o_stride = o_stride;
    p.q_stride = q_stride;
    p.heads = nheads;
    p.group = group;
    p.tile_tokens = kTileRows / group;
    // no context is longer than its block table: such a window hides nothing, and those
    // left are below 2^30, so that a position less a window stays in 32 bits
    p.window = window >= static_cast<int64_t>(table_width) * page_size ? 0 : window;
    // a scale of zero still has to leave the hidden keys' -infinity as it is
    p.scale_log2 = std::fmax(scale_log2, 0x1p-120f);
    p.negate = softmax_scale < 0.f;
    p.seq_units = reinterpret_cast<int32_t *>(ws + L.seq_units);
    for (int k = 0; k < 2; ++k)
        p.line[k] = AttnLine{reinterpret_cast<AttnUnit *>(ws + L.units[k]),
                             reinterpret_cast<AttnPiece *>(ws + L.pieces[k]),
                             reinterpret_cast<int64_t *>(ws + L.cum[k]),
                             reinterpret_cast<float *>(ws + L.part_o[k]),
                             reinterpret_cast<float2 *>(ws + L.part_ml[k]),
                             reinterpret_cast<int4 *>(ws + L.split[k])};

    AttnMaps m = {};
    const uint64_t D = head_dim, rows = static_cast<uint64_t>(num_pages) * nheads_kv;
    const uint32_t box = page_size < kTileKeys ? page_size : kTileKeys;
    bool ok = make_map(&m.Q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, q, D, nheads, total_len, D * 2,
                       q_stride * 2, 64, group, p.tile_tokens, CU_TENSOR_MAP_SWIZZLE_128B);
    for (int kv = 0; kv < 2 && ok; ++kv) {
        CUtensorMap *t = kv ? &m.V : &m.K;
        const void *base = kv ? v_cache : k_cache;
        if (cache_type == SSD_KV_BF16) {
            ok = make_map(t, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, D, page_size, rows, D * 2,
                          D * 2 * page_size, 64, box, 1, CU_TENSOR_MAP_SWIZZLE_128B);
        } else {
            ok = make_map(t, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, D, page_size, rows, D,
                          D * page_size, head_dim, box, 1, CU_TENSOR_MAP_SWIZZLE_NONE);
        }
    }
    if (!ok)
        return SSD_ERR_CUDA;

    // a unit has at most min(total_len, 2 tiles' tokens) tokens and at least one:
    // what that rules out is not launched
    const bool tiles = std::min<int64_t>(total_len, 2 * p.tile_tokens) * group > kFewRows;
    const bool few = group <= kFewRows;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    cudaError_t e = launch_pdl(attn_plan_kernel, dim3(kPlanCtas),
                               batch <= kPlanSmall ? kPlanSmall : kPlanThreads, stream, p);
    const bool bf16 = cache_type == SSD_KV_BF16, fp8 = cache_type == SSD_KV_FP8_E4M3;
    if (e == cudaSuccess && tiles)
        e = bf16 ? launch_attn_bf16(p, m, stream)
                 : fp8 ? launch_attn_fp8(p, m, stream) : launch_attn_int8(p, m, stream);
    if (e == cudaSuccess && few)
        e = bf16 ? launch_attn_few_bf16(p, stream)
                 : fp8 ? launch_attn_few_fp8(p, stream) : launch_attn_few_int8(p, stream);
    if (e == cudaSuccess) {
        const dim3 grid(kJoinCtas);
        e = head_dim == 128 ? launch_pdl(attn_join_kernel<128>, grid, kJoinWarps * 32, stream, p)
                            : launch_pdl(attn_join_kernel<64>, grid, kJoinWarps * 32, stream, p);
    }
    return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
