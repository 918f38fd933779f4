"""The short causal convolution on the GPU against the formula in 64 bits.

Bound of y, with S = |bias| + sum |w u| and v the sum: W fused products and adds in
fp32 are off by at most 2 W 2^-24 S; silu changes that by at most 1.1.  Its e^-v is
off by 2^-22 + |v| 2^-23 relative (argument and function), the quotient by 2^-22, and
quotients below 2^-126 |v| are zero.  y is rounded to bf16 once."""
from __future__ import annotations

import numpy as np
import pytest

from layer_helpers import E, U, Ragged, f64, near, same_bits, sliced

pytestmark = pytest.mark.gpu


def conv_ref(r, x, weight, bias, pool, silu):
    """y (NaN where no row is written), its bound, the pool after the call."""
    w = weight.shape[1]
    y, bound, pool = np.full(x.shape, np.nan), np.zeros(x.shape), pool.copy()
    for _, lo, hi, slot, has in r.each():
        before = pool[slot] if has else np.zeros((w - 1, x.shape[1]))
        line = np.concatenate([before, x[lo:hi]])
        n = hi - lo
        v, s = np.zeros((n, x.shape[1])), np.zeros((n, x.shape[1]))
        v, s = v + bias, s + np.abs(bias)
        for j in range(w):
            v, s = v + line[j:j + n] * weight[:, j], s + np.abs(line[j:j + n] * weight[:, j])
        b = 2 * w * E * s
        if silu:
            out = v / (1 + np.exp(-v))
            b = 1.1 * b + np.abs(out) * (2.0 ** -21 + np.abs(v) * 2.0 ** -23) + 2.0 ** -126 * (1 + np.abs(v))
        else:
            out = v
        y[lo:hi], bound[lo:hi] = out, U * np.abs(out) + b * (1 + U) + 2.0 ** -133
        if slot >= 0:
            pool[slot] = line[n:]
    return y, bound, pool


def run(r, channels, width, silu=True, bias=True, seed=0, strided=False, stream=None, change=None):
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    g = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g)

    x = normal(r.rows, channels).bfloat16().cuda()
    weight, b = normal(channels, width).cuda(), normal(channels).cuda() if bias else None
    pool = normal(r.slots, width - 1, channels).bfloat16().cuda()
    y = torch.full_like(x, 7.0)
    if change:
        change(x, pool)
    before = pool.clone()
    xs, ys = x, y
    if strided:
        wide_x, xs = sliced(x)
        wide_y, ys = sliced(y)
        kept = wide_x.clone(), wide_y.clone()
    pkg.ssd_causal_conv_varlen_fwd(ys, xs, weight, b, pool, *r.where, silu=silu, errors=r.errors,
                                   stream=stream)
    torch.cuda.synchronize()
    if strided:
        assert same_bits(kept[0], wide_x)
        kept[1][:, 16:-16] = ys
        assert same_bits(kept[1], wide_y)
    want, bound, pool_ref = conv_ref(r, f64(x), f64(weight), f64(b) if bias else np.zeros(channels),
                                     f64(before), silu)
    got = f64(ys)
    end = int(r.start[-1])
    assert (got[end:] == 7.0).all()          # rows behind the last sequence
    near(got[:end], want[:end], bound[:end], "y")
    assert np.array_equal(f64(pool), pool_ref, equal_nan=True)
    assert r.errors.item() == 0
    return ys, pool


LENS = [
    [1], [0], [5], [33], [300], [1] * 40, [0, 1, 2, 3, 4, 5, 0, 0, 31, 32, 33, 1, 1, 64, 65, 0],
    [2] * 100 + [97] + [0] * 70 + [3], [1000, 1, 999], [31, 1, 30, 2, 29, 3, 0, 28],
]


@pytest.mark.parametrize("lens", range(len(LENS)))
@pytest.mark.parametrize("width", [2, 3, 4])
def test_against_the_formula(lens, width):
    run(Ragged(LENS[lens], seed=lens), 264, width, seed=lens)


@pytest.mark.parametrize("channels", [8, 248, 256, 520, 4352])
@pytest.mark.parametrize("silu,bias", [(True, False), (False, True), (False, False)])
def test_channels_and_options(channels, silu, bias):
    run(Ragged([70, 1, 0, 2], seed=1), channels, 4, silu, bias)


def test_strided_and_padded():
    """Column slices, rows behind the last sequence, sequences without a slot."""
    run(Ragged([40, 1, 3, 0], seed=2, rows=100, none=(1, 3)), 272, 4, strided=True)
    run(Ragged([0, 0], seed=2, rows=33), 64, 3, strided=True)


def test_large_values():
    """Infinities and NaN reach their window alone; silu of far values."""
    import torch

    def change(x, pool):
        x[10, :32] = float("inf")
        x[20, 32:64] = float("nan")
        x[41, :64] = -float("inf")
        x[60:, :] *= 1e30
        pool[:, 0, 100] = float("nan")
    run(Ragged([40, 2, 0, 60], seed=3), 128, 4, change=change)
    run(Ragged([40, 2, 0, 60], seed=3), 128, 4, silu=False, change=change)


def test_steps_equal_one_prompt():
    """A prompt in parts and single tokens gives the prompt's rows and slot, bit for bit."""
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    g = torch.Generator().manual_seed(4)
    n, c, w = 83, 328, 4
    x = torch.randn(n, c, generator=g).bfloat16().cuda()
    weight, bias = torch.randn(c, w, generator=g).cuda(), torch.randn(c, generator=g).cuda()
    slot = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = []
    for cuts in ([0, n], [0, 1, 2, 34, 35, 36, 80, 81, 82, n]):
        y, pool = torch.empty_like(x), torch.full((1, w - 1, c), 3.0, dtype=torch.bfloat16, device="cuda")
        for lo, hi in zip(cuts, cuts[1:]):
            pkg.ssd_causal_conv_varlen_fwd(
                y[lo:hi], x[lo:hi], weight, bias, pool,
                torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda"),
                torch.tensor([lo > 0], device="cuda"), slot)
        out.append((y, pool))
    assert same_bits(out[0][0], out[1][0]) and same_bits(out[0][1], out[1][1])


def test_device_side_errors():
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    from mamba_ssd_chunked_varlen_gb300 import binding
    x = torch.randn(20, 64, device="cuda").bfloat16()
    weight = torch.randn(64, 4, device="cuda")
    for offsets in ([0, 8, 4, 20], [1, 8, 9, 20], [0, 8, 9, 21], [0, -3, 9, 20]):
        y, pool = torch.empty_like(x), torch.zeros(6, 3, 64, dtype=torch.bfloat16, device="cuda")
        errors = torch.zeros(1, dtype=torch.int32, device="cuda")
        pkg.ssd_causal_conv_varlen_fwd(
            y, x, weight, None, pool, torch.tensor(offsets, dtype=torch.int32, device="cuda"), None,
            torch.arange(3, dtype=torch.int32, device="cuda"), errors=errors)
        assert errors.item() == binding.DEVERR_BAD_QUERY_START_LOC
        assert not pool[3:].any()
    r = Ragged([8, 5, 7], seed=5)
    y, pool = torch.empty_like(x), torch.randn(r.slots, 3, 64, device="cuda").bfloat16()
    z, kept = torch.empty_like(x), pool.clone()
    pkg.ssd_causal_conv_varlen_fwd(y, x, weight, None, pool, *r.where, errors=r.errors)
    assert r.errors.item() == 0
    r.cache_indices[1] = r.slots
    other = kept.clone()
    pkg.ssd_causal_conv_varlen_fwd(z, x, weight, None, other, *r.where, errors=r.errors)
    assert r.errors.item() == binding.DEVERR_BAD_CACHE_INDEX
    slot = int(r.slot[1])
    assert same_bits(other[slot], kept[slot])
    other[slot] = pool[slot]
    assert same_bits(other, pool) and same_bits(z[:8], y[:8]) and same_bits(z[16:], y[16:])


def test_stream_and_graph():
    """On a stream of its own, and captured: a replay takes the buffers' new contents."""
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    r = Ragged([37, 1, 4], seed=6)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    run(r, 264, 4, stream=stream)
    x = torch.randn(r.rows, 264, device="cuda").bfloat16()
    weight = torch.randn(264, 4, device="cuda")
    y, pool = torch.empty_like(x), torch.zeros(r.slots, 3, 264, dtype=torch.bfloat16, device="cuda")

    def call(y, pool):
        pkg.ssd_causal_conv_varlen_fwd(y, x, weight, None, pool, *r.where, errors=r.errors)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(y, pool)
    for seed in range(2):
        x.copy_(torch.randn(r.rows, 264, generator=torch.Generator().manual_seed(seed)))
        want, kept = torch.empty_like(y), pool.clone()
        graph.replay()
        call(want, kept)
        torch.cuda.synchronize()
        assert same_bits(y, want) and same_bits(pool, kept)


def test_far_rows():
    """Rows past 2^31 elements."""
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    wide, n = 1 << 20, 2100
    buffer = torch.zeros(n, wide, dtype=torch.bfloat16, device="cuda")
    x, y = buffer[:, 64:128], buffer[:, 256:320]
    x.copy_(torch.randn(n, 64, generator=torch.Generator().manual_seed(7)))
    weight = torch.randn(64, 4, device="cuda")
    pool = torch.zeros(1, 3, 64, dtype=torch.bfloat16, device="cuda")
    where = torch.tensor([0, n], dtype=torch.int32, device="cuda"), None, \
        torch.zeros(1, dtype=torch.int32, device="cuda")
    pkg.ssd_causal_conv_varlen_fwd(y, x, weight, None, pool, *where)
    near_x, near_y = x.contiguous(), torch.empty(n, 64, dtype=torch.bfloat16, device="cuda")
    pkg.ssd_causal_conv_varlen_fwd(near_y, near_x, weight, None, pool, *where)
    assert same_bits(y, near_y)


def test_far_slots():
    """A slot past 2^31 elements."""
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    channels = 1 << 20
    slots = (1 << 31) // (3 * channels) + 3
    pool = torch.zeros(slots, 3, channels, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(8)
    x, old = (torch.randn(n, channels, generator=g, device="cuda").bfloat16() for n in (2, 3))
    weight = torch.randn(channels, 4, generator=g, device="cuda")
    where = torch.tensor([0, 2], dtype=torch.int32, device="cuda"), torch.tensor([True], device="cuda")
    out = []
    for p, slot in ((pool, slots - 1), (torch.zeros(1, 3, channels, dtype=torch.bfloat16, device="cuda"), 0)):
        p[slot] = old
        y = torch.empty_like(x)
        pkg.ssd_causal_conv_varlen_fwd(y, x, weight, None, p, *where,
                                       torch.tensor([slot], dtype=torch.int32, device="cuda"))
        out.append((y, p[slot]))
    assert same_bits(out[0][0], out[1][0]) and same_bits(out[0][1], out[1][1])
    assert not pool[:-1].any()
