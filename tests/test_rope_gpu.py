"""Rotary positions on the GPU, alone and with the cache's write, against the formula:
angles from integers of 128 bits, cosine, sine and products in 64.

Bound before the output's rounding: the angle is off by 2^-33 + 2^-34 turns (its table
and the 32 bits kept) and its rounding to fp32, 2^-24 of half a turn: 2^-22 in all, in
radians; the functions are off by 2^-22 at most; magnitude, products and the sum are four
roundings.  So |y| is off by at most m (|a| + |b|) (2^-21 + 4 2^-24) < m (|a| + |b|) 2^-20."""
from __future__ import annotations

import functools

import numpy as np
import pytest

from attn_helpers import TINY, TOP, Batch
from layer_helpers import E, U, f64, near, same_bits, sliced

pytestmark = pytest.mark.gpu

OFF = 2.0 ** -20


@functools.lru_cache(None)
def inverse_two_pi(bits=400):
    """floor(2^bits / (2 pi)), pi by Machin's arctangents."""
    def arctan_inverse(x, one):
        total = term = one // x
        n, sign = 3, -1
        while term:
            term //= x * x
            total += sign * (term // n)
            n, sign = n + 2, -sign
        return total
    one = 1 << (2 * bits)
    pi = 4 * (4 * arctan_inverse(5, one) - arctan_inverse(239, one))
    return (1 << (3 * bits)) // (2 * pi)


def turns_of(frequencies):
    """The frequencies as integers of 2^-128 turns."""
    out = []
    for f in frequencies:
        n, d = float(f).as_integer_ratio()
        out.append(n * inverse_two_pi() // d >> (400 - 128))
    return out


def angles(positions, frequencies):
    """Angles in radians within a turn, (positions, frequencies)."""
    table = turns_of(frequencies)
    mask = (1 << 128) - 1
    return np.array([[2 * np.pi * ((int(p) * t & mask) / 2.0 ** 128) for t in table] for p in positions])


def rotate_ref(x, angle, part, neighbours, m):
    """Rotated heads in 64 bits and the bound of the module docstring."""
    y, off = x.copy(), np.zeros_like(x)
    cos, sin = m * np.cos(angle)[:, None], m * np.sin(angle)[:, None]
    at = (slice(0, part, 2), slice(1, part, 2)) if neighbours else (slice(0, part // 2), slice(part // 2, part))
    a, b = x[..., at[0]], x[..., at[1]]
    y[..., at[0]], y[..., at[1]] = a * cos - b * sin, b * cos + a * sin
    for i in at:
        off[..., i] = abs(m) * (np.abs(a) + np.abs(b)) * OFF
    return y, off


def positions_of(lens):
    return np.concatenate([np.arange(kv - n, kv) for n, kv in lens] + [np.zeros(0)]).astype(np.int64)


def make(lens, heads, kv_heads, dim, seed=0):
    import torch
    g = torch.Generator().manual_seed(seed)
    total = sum(n for n, _ in lens)
    start = np.concatenate([[0], np.cumsum([n for n, _ in lens])])
    q, k = (torch.randn(total, h, dim, generator=g).bfloat16().cuda() for h in (heads, kv_heads))
    return q, k, torch.tensor(start, dtype=torch.int32, device="cuda"), \
        torch.tensor([kv for _, kv in lens], dtype=torch.int32, device="cuda")


FAR = [(3, 1 << 20), (2, (1 << 31) - 1), (5, 5), (1, 1000001)]
SHAPES = [
    # lens, q heads, kv heads, dim, rotated part
    ([(1, 1)], 1, 1, 64, 64),
    ([(1, 17), (3, 3), (0, 9), (16, 33)], 6, 2, 128, 128),
    (FAR, 5, 3, 128, 128),
    (FAR, 4, 4, 64, 16),
    ([(33, 5000)], 32, 8, 128, 32),
    ([(7, 70000), (1, 1)], 3, 1, 64, 48),
    ([(9, 9)], 8, 8, 128, 112),
]


@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_rotation(shape, neighbours):
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    lens, heads, kv_heads, dim, part = SHAPES[shape]
    q, k, start, kv_lens = make(lens, heads, kv_heads, dim, shape)
    freqs, m = pkg.rope_frequencies(part, scaling="ramp", factor=3.0)
    table = pkg.alloc_rope_table(freqs)
    errors = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = torch.zeros_like(q), torch.zeros_like(k)
    pkg.ssd_rope_varlen_fwd(outs[0], q, outs[1], k, table, start, kv_lens, interleaved=neighbours,
                            magnitude=m, errors=errors)
    assert errors.item() == 0
    angle = angles(positions_of(lens), freqs)
    for x, y in zip((q, k), outs):
        want, off = rotate_ref(f64(x), angle, part, neighbours, m)
        near(f64(y), want, U * np.abs(want) + off * (1 + U), "rotated")
        assert same_bits(y[..., part:], x[..., part:])
    # one of them alone, in place
    for x, y, alone in zip((q, k), outs, (lambda t: (t, t, None, None), lambda t: (None, None, t, t))):
        z = x.clone()
        pkg.ssd_rope_varlen_fwd(*alone(z), table, start, kv_lens, interleaved=neighbours, magnitude=m)
        assert same_bits(z, y)


def test_table():
    """The table's entries are the frequencies in turns, to the last bit but one."""
    import mamba_ssd_chunked_varlen_gb300 as pkg
    freqs = pkg.rope_frequencies(128, 500000.0)[0] + [0.0, 1e-300, 2.0 ** -64, 2.0 ** -70, 3.0, 6.283185307179585]
    got = pkg.alloc_rope_table(freqs, "cpu").tolist()
    for t, want in zip(got, turns_of(freqs)):
        assert abs((t % (1 << 64) << 64) - want) <= 0.75 * 2 ** 64, (t, want)


def test_many_tokens_equal_few():
    """More tokens than spread a token's rows over warps: the same bits."""
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    lens = [(1700, 1700), (1, 40), (1200, 1300)]
    q, k, start, kv_lens = make(lens, 5, 3, 64, 1)
    table = pkg.alloc_rope_table(pkg.rope_frequencies(64)[0])
    whole = torch.empty_like(q), torch.empty_like(k)
    pkg.ssd_rope_varlen_fwd(whole[0], q, whole[1], k, table, start, kv_lens)
    parts, at = (torch.empty_like(q), torch.empty_like(k)), 0
    for n, kv in lens:
        s = slice(at, at + n)
        pkg.ssd_rope_varlen_fwd(parts[0][s], q[s], parts[1][s], k[s], table,
                                torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                                torch.tensor([kv], dtype=torch.int32, device="cuda"))
        at += n
    assert same_bits(whole[0], parts[0]) and same_bits(whole[1], parts[1])


CACHES = [
    # lens, q heads, kv heads, dim, page, rotated part
    ([(1, 1)], 1, 1, 64, 16, 64),
    ([(1, 17), (3, 3), (0, 9), (16, 33)], 4, 2, 128, 16, 128),
    ([(5, 300), (130, 130), (1, 257)], 9, 3, 64, 64, 32),
    ([(129, 400)], 8, 8, 128, 256, 96),
    ([(2, 2)] * 40 + [(0, 0)] * 3 + [(1, 50)] * 33, 5, 5, 128, 32, 128),
    ([(1500, 1500), (1000, 1111)], 2, 1, 64, 128, 64),
]


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("shape", range(len(CACHES)))
def test_write(shape, kind):
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    lens, heads, kv_heads, dim, page, part = CACHES[shape]
    neighbours = shape % 2 == 1
    b = Batch(lens, heads, kv_heads, dim, page, kind, seed=shape)
    cut = [(x[kv - n:], y[kv - n:]) for (n, kv), x, y in zip(lens, b.k_seq, b.v_seq)]
    k, v = torch.cat([x for x, _ in cut]).cuda(), torch.cat([y for _, y in cut]).cuda()
    freqs, m = pkg.rope_frequencies(part, scaling="linear", factor=2.0)[0], 1.25
    table = pkg.alloc_rope_table(freqs)
    other = [None if t is None else t.clone() for t in b.cache]
    q_out, k_out = torch.zeros_like(b.q), torch.zeros_like(k)
    pkg.ssd_rope_kv_cache_write(q_out, b.q, k, v, table, *b.cache, *b.where, interleaved=neighbours,
                                magnitude=m, errors=b.errors)
    # the queries, the values and a bf16 cache as by the two calls, to the bit
    q_two = torch.zeros_like(b.q)
    pkg.ssd_rope_varlen_fwd(q_two, b.q, k_out, k, table, *b.where[:2], interleaved=neighbours, magnitude=m)
    assert same_bits(q_out, q_two)
    pkg.ssd_kv_cache_write(k_out, v, *other, *b.where)
    pairs = list(zip(b.cache, other))
    for x, y in pairs if kind == "bf16" else (pairs[1], pairs[3]):
        assert y is None or same_bits(x, y)
    assert b.errors.item() == 0
    if kind == "bf16":
        return
    want, off = rotate_ref(f64(k), angles(positions_of(lens), freqs), part, neighbours, m)
    at, owned = 0, torch.zeros(b.pages, page, dtype=torch.bool)
    for s, (n, kv) in enumerate(lens):
        j = torch.arange(kv - n, kv)
        pages, rows = b.table_cpu[s].long()[j // page], j % page
        owned[pages, rows] = True
        code = f64(b.k_cache.float()[pages.cuda(), :, rows.cuda()])
        scale = f64(b.k_scale[pages.cuda(), :, rows.cuda()])
        w, o = want[at:at + n], off[at:at + n]
        a = np.maximum(np.abs(w).max(-1), TINY)
        near(scale, a / TOP[kind], (o.max(-1) + a * 2 * E) / TOP[kind], "scale")
        step = 1.0 if kind == "int8" else np.maximum(2.0 ** -9, np.abs(code) * 2.0 ** -3)
        near(code * scale[..., None], w, 0.5 * step * scale[..., None] * (1 + 2.0 ** -6) + 2 * o, "k")
        at += n
    # rows that no new token has are as they were
    keep = ~owned.cuda()
    for x, y in (pairs[0], pairs[2]):
        same = (x.view(torch.uint8) == y.view(torch.uint8)).view(b.pages, kv_heads, page, -1).all(-1).all(1)
        assert same[keep].all()


@pytest.mark.parametrize("kind", ["fp8", "int8"])
def test_codes_of_extreme_rows(kind):
    """Rows with infinities and NaN read back as NaN, and no other; zeros as zeros."""
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    b = Batch([(12, 12)], 2, 2, 64, 16, kind, seed=5)
    k, v = b.k_seq[0].cuda(), b.v_seq[0].cuda()
    k[0] = 0.0
    k[2, :, 3] = 1e38
    k[3, 0, 9] = float("inf")
    k[4, 1, 63] = float("nan")
    v[5, 0, 0] = -float("inf")
    k[6] *= 2.0 ** -80
    pkg.ssd_rope_kv_cache_write(torch.empty_like(b.q), b.q, k, v, pkg.alloc_rope_table(pkg.rope_frequencies(64)[0]),
                                *b.cache, *b.where, errors=b.errors)
    rk, rv = torch.empty_like(k), torch.empty_like(v)
    pkg.ssd_kv_cache_read(rk, rv, *b.cache, *b.where, errors=b.errors)
    bad = torch.zeros(2, 12, 2, dtype=torch.bool, device="cuda")
    bad[0, 3, 0] = bad[0, 4, 1] = bad[1, 5, 0] = True
    for t, x in zip(bad, (rk, rv)):
        assert torch.equal(torch.isnan(x).all(-1), t) and torch.equal(torch.isnan(x).any(-1), t)
    assert (rk[0] == 0).all() and b.errors.item() == 0


def test_strided_padded_and_left_alone():
    """Column slices; rows at a negative position, behind the last sequence or of a
    missing page are left as they were."""
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    from mamba_ssd_chunked_varlen_gb300 import attention, binding
    b = Batch([(6, 40), (20, 33)], 4, 2, 64, 16, "int8", seed=6)
    total = 30      # four rows more than the sequences'
    wide = torch.randn(total, 8 * 64 + 24, device="cuda").bfloat16()
    q, k, v = wide[:, 8:264].view(total, 4, 64), wide[:, 272:400].view(total, 2, 64), \
        wide[:, 400:528].view(total, 2, 64)
    table = pkg.alloc_rope_table(pkg.rope_frequencies(32)[0])
    want = torch.zeros(total, 4, 64, dtype=torch.bfloat16, device="cuda")
    other = [t.clone() for t in b.cache]
    pkg.ssd_rope_kv_cache_write(want[:26], q[:26].contiguous(), k[:26].contiguous(), v[:26].contiguous(), table,
                                *other, *b.where)
    out_wide, out = sliced(torch.full((total, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda"))
    kept = wide.clone(), out_wide.clone()
    pkg.ssd_rope_kv_cache_write(out, q, k, v, table, *b.cache, *b.where, errors=b.errors)
    assert b.errors.item() == 0 and same_bits(wide, kept[0])
    assert same_bits(out[:26], want[:26]) and (out[26:] == 7.0).all()
    kept[1][:, 16:-16] = out.flatten(1)
    assert same_bits(out_wide, kept[1])
    for x, y in zip(b.cache, other):
        assert same_bits(x, y)
    # the first sequence's first four rows are padding; the second's first page is missing
    b.kv_lens[0] = 2
    b.block_table[1, 0] = -1
    out.fill_(7.0)
    before = [t.clone() for t in b.cache]
    pkg.ssd_rope_kv_cache_write(out, q + 1, k + 1, v + 1, table, *b.cache, *b.where, errors=b.errors)
    assert b.errors.item() == attention.DEVERR_BAD_PAGE
    assert (out[:4] == 7.0).all() and (out[26:] == 7.0).all() and (out[4:26] != 7.0).any(-1).any(-1).all()
    changed = torch.zeros(b.pages, 16, dtype=torch.bool, device="cuda")
    for x, y in zip(before, b.cache):
        diff = (x.view(torch.uint8) != y.view(torch.uint8)).view(b.pages, 2, 16, -1)
        changed |= diff.any(-1).any(1)
    rows = torch.zeros_like(changed)
    for s, j in [(0, 0), (0, 1)] + [(1, j) for j in range(16, 33)]:
        rows[b.row_of(s, j)] = True
    assert torch.equal(changed, rows)
    # lengths and offsets that are none
    for change, flag in ((lambda: b.kv_lens.__setitem__(0, -1), attention.DEVERR_BAD_KV_LEN),
                         (lambda: b.query_start_loc.__setitem__(1, 40), binding.DEVERR_BAD_QUERY_START_LOC)):
        b = Batch([(6, 40), (20, 33)], 4, 2, 64, 16, "int8", seed=6)
        change()
        out.fill_(7.0)
        pkg.ssd_rope_varlen_fwd(out, q, None, None, table, *b.where[:2], errors=b.errors)
        assert b.errors.item() == flag and (out[:6] == 7.0).all()


def test_stream_and_graph():
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    b = Batch([(3, 40), (1, 33)], 4, 2, 64, 16, "fp8", seed=7)
    k, v = (torch.randn(4, 2, 64, device="cuda").bfloat16() for _ in range(2))
    table = pkg.alloc_rope_table(pkg.rope_frequencies(64)[0])
    out = torch.empty_like(b.q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.ssd_rope_kv_cache_write(out, b.q, k, v, table, *b.cache, *b.where, errors=b.errors)
    stream = torch.cuda.Stream()
    for step in range(2):
        b.kv_lens -= step          # the captured call goes by the lengths of the replay
        want, other = torch.empty_like(out), [t.clone() for t in b.cache]
        torch.cuda.synchronize()
        pkg.ssd_rope_kv_cache_write(want, b.q, k, v, table, *other, *b.where, stream=stream)
        graph.replay()
        torch.cuda.synchronize()
        assert same_bits(out, want) and all(same_bits(x, y) for x, y in zip(b.cache, other))
    assert b.errors.item() == 0


def test_far_pages_and_rows():
    """A cache row past 2^31 elements, and rows of q past 2^31 elements."""
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    pages = (1 << 31) // (256 * 2 * 64) + 3
    caches = [torch.zeros((pages, 2, 256, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    k = torch.randn(300, 2, 64, device="cuda").bfloat16()
    where = (torch.tensor([0, 300], dtype=torch.int32, device="cuda"),
             torch.tensor([300], dtype=torch.int32, device="cuda"),
             torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda"))
    table = pkg.alloc_rope_table(pkg.rope_frequencies(64)[0])
    wide = torch.zeros(300, 1 << 23, dtype=torch.bfloat16, device="cuda")
    q = wide[:, 1024:1152].view(300, 2, 64)
    q.copy_(k)
    q_out = torch.empty_like(k)
    pkg.ssd_rope_kv_cache_write(q_out, q, k, k, table, *caches, None, None, *where)
    want = torch.empty_like(k)
    pkg.ssd_rope_varlen_fwd(want, k, None, None, table, *where[:2])
    assert same_bits(q_out, want)
    assert same_bits(caches[0][pages - 1].transpose(0, 1), want[:256])
    assert same_bits(caches[1][pages - 2, :, :44].transpose(0, 1), k[256:])
    assert not caches[0][:pages - 2].any()
