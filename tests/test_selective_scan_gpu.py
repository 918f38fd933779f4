"""The selective scan on the GPU against the recurrence in 64 bits.

The bound runs along with the recurrence.  The step d = softplus(v) is off by
2^-21 + |v| 2^-23 + 2^-24 relative: v's own rounding, the exponential (argument and function,
2^-22 and |v| 2^-24) and the logarithm's polynomial (2^-22).  A decay exp(d A) is off by
|d A| (the step's error + 2^-22) + 2^-22 + 2^-24 relative, an input d x B by the step's error
and two roundings, and every step rounds h once:

    off(h') = a off(h) + a |h| err(a) + |d x B| err(in) + 2^-24 |h'|

y adds N + 2 roundings of sum |C h| + |D x|, the gate 2^-21 + |z| 2^-23 and a rounding, and
bf16 half a step."""
from __future__ import annotations

import numpy as np
import pytest

from layer_helpers import E, U, Ragged, f64, near, same_bits, sliced

pytestmark = pytest.mark.gpu


def scan_ref(r, v, pool, softplus, bf16):
    """y, its bound, the pool after the call and its bound."""
    x, dt, A, B, C, D, z, bias = (v[k] for k in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias"))
    raw = dt + bias
    d = np.logaddexp(0.0, raw) if softplus else raw
    err_d = 2.0 ** -21 + np.abs(raw) * 2.0 ** -23 + E if softplus else np.full_like(raw, E)
    if not softplus:     # the sum's rounding is relative to it
        err_d = err_d + 0.0
    y, yb = np.full(x.shape, np.nan), np.zeros(x.shape)
    pool, pb = pool.copy(), np.zeros_like(pool)
    n = A.shape[1]
    for _, lo, hi, slot, has in r.each():
        h = pool[slot].copy() if has else np.zeros_like(A)
        off = np.zeros_like(h)
        for t in range(lo, hi):
            arg = d[t][:, None] * A
            a = np.exp(arg)
            inp = (d[t] * x[t])[:, None] * B[t]
            e = err_d[t][:, None]
            new = a * h + inp
            off = a * off + a * np.abs(h) * (np.abs(arg) * (e + 2.0 ** -22) + 2.0 ** -22 + E) \
                + np.abs(inp) * (e + 2 * E) + E * np.abs(new) + 2.0 ** -126
            h = new
            out = h @ C[t] + D * x[t]
            b = off @ np.abs(C[t]) + (n + 2) * E * (np.abs(h) @ np.abs(C[t]) + np.abs(D * x[t]))
            if z is not None:
                g = z[t] / (1 + np.exp(-z[t]))
                b = np.abs(g) * b + np.abs(out * g) * (2.0 ** -21 + np.abs(z[t]) * 2.0 ** -23 + E)
                out = out * g
            y[t], yb[t] = out, b * (1 + U) + U * np.abs(out) + 2.0 ** -126
        if slot >= 0:
            pool[slot], pb[slot] = h, off + (U * np.abs(h) + U * off + 2.0 ** -133 if bf16 else 0.0)
    return y, yb, pool, pb


def make(r, channels, dstate, seed=0, gate=True, bf16=False, D=True, bias=True, softplus=True):
    import torch
    g = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g)

    raw = 0.5 * normal(r.rows, channels)
    v = dict(x=normal(r.rows, channels), dt=raw if softplus else 0.1 * raw.abs(), B=normal(r.rows, dstate),
             C=normal(r.rows, dstate), z=2 * normal(r.rows, channels) if gate else None)
    v = {k: None if t is None else t.bfloat16().cuda() for k, t in v.items()}
    v["A"] = -(torch.rand(channels, dstate, generator=g) * dstate + 0.5).cuda()
    v["D"] = normal(channels).cuda() if D else None
    u = torch.exp(torch.rand(channels, generator=g) * np.log(100.0) + np.log(1e-3))
    v["dt_bias"] = (torch.log(torch.expm1(u)) if softplus else u).cuda() if bias else None
    v["pool"] = normal(r.slots, channels, dstate).to(torch.bfloat16 if bf16 else torch.float32).cuda()
    return v


def call(r, v, y, pool, softplus=True, stream=None, workspace=None):
    import mamba_ssd_chunked_varlen_gb300 as pkg
    if workspace is None:
        workspace = pkg.alloc_selective_scan_workspace(r.rows, len(r.lens), *v["A"].shape)
    pkg.ssd_selective_scan_varlen_fwd(y, v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], v["z"], v["dt_bias"], pool,
                                      *r.where, dt_softplus=softplus, workspace=workspace, errors=r.errors,
                                      stream=stream)


def check(r, channels, dstate, seed=0, softplus=True, change=None, strided=False, stream=None, **options):
    import torch
    v = make(r, channels, dstate, seed, softplus=softplus, **options)
    if change:
        change(v)
    y, pool = torch.full_like(v["x"], 7.0), v["pool"].clone()
    use = dict(v)
    if strided:
        kept = {}
        for k in ("x", "dt", "B", "C", "z"):
            if v[k] is not None:
                wide, use[k] = sliced(v[k], 8)
                kept[k] = wide, wide.clone()
        wide_y, y = sliced(y, 8)
        before = wide_y.clone()
    torch.cuda.synchronize()
    call(r, use, y, pool, softplus, stream)
    torch.cuda.synchronize()
    if strided:
        assert all(same_bits(a, b) for a, b in kept.values())
        before[:, 8:-8] = y
        assert same_bits(before, wide_y)
    ref = {k: f64(t) if t is not None else None for k, t in v.items()}
    for k in ("D", "dt_bias"):
        ref[k] = np.zeros(channels) if ref[k] is None else ref[k]
    bf16 = pool.dtype == torch.bfloat16
    want, bound, pool_ref, pool_bound = scan_ref(r, ref, f64(v["pool"]), softplus, bf16)
    end, got = int(r.start[-1]), f64(y)
    assert (got[end:] == 7.0).all()
    near(got[:end], want[:end], bound[:end], "y")
    named = sorted(s for s in set(r.slot) if s >= 0)
    near(f64(pool)[named], pool_ref[named], pool_bound[named], "pool")
    rest = [s for s in range(r.slots) if s not in named]
    assert same_bits(pool[rest], v["pool"][rest])
    assert r.errors.item() == 0
    return y, pool


LENS = [
    [1], [0], [7], [8], [33], [300], [1] * 20, [0, 1, 2, 3, 0, 9, 31, 32, 33, 8, 16, 0, 65],
    [129, 1, 40], [2] * 30 + [70] + [0] * 40 + [3],
]


@pytest.mark.parametrize("lens", range(len(LENS)))
@pytest.mark.parametrize("dstate", [8, 16, 32, 64])
def test_against_the_recurrence(lens, dstate):
    check(Ragged(LENS[lens], seed=lens), 72, dstate, seed=lens)


# sequences that are cut into chunks: of 64 tokens, the shortest there are, or more
@pytest.mark.parametrize("lens,channels,dstate", [
    ([128], 8, 8), ([127], 8, 16), ([129], 40, 16), ([1000], 8, 16), ([1000, 3, 700, 1, 129, 0, 128, 127], 72, 16),
    ([64] * 9 + [192, 0, 193], 72, 32), ([1, 500, 1, 1, 300], 24, 64), ([1500], 1024, 16), ([700, 600], 2048, 16),
    ([2000, 1500, 40, 1900], 264, 8),
])
def test_chunks(lens, channels, dstate):
    check(Ragged(lens, seed=len(lens)), channels, dstate, seed=dstate, gate=dstate != 32)
    check(Ragged(lens, seed=len(lens) + 1, rows=sum(lens) + 70, none=(0,)), channels, dstate, bf16=True)


# batches of few tokens with a longer sequence, and of more sequences than a plan's or a CTA's
# threads
@pytest.mark.parametrize("lens", [[101, 60], [32, 128], [15, 161], [200, 0], [50, 33, 101, 17]])
@pytest.mark.parametrize("dstate", [8, 16, 32, 64])
def test_many_channels_in_whole_sequences(lens, dstate):
    """So many warps a sequence that nothing is cut: two sequences are two CTAs an SM at
    most, four of them more."""
    check(Ragged(lens, seed=dstate), 104_960 // dstate, dstate, seed=len(lens), gate=dstate != 8,
          bf16=dstate == 32)


@pytest.mark.parametrize("lens", [[1, 8, 9, 2, 40, 0, 1, 1, 1], [8] * 5, [9, 8, 7, 1, 1], [3] * 70 + [200] + [1] * 30,
                                  [0] * 30 + [25], [3] * 600 + [150, 0, 1, 9], [1, 20] * 300])
def test_few_tokens(lens):
    check(Ragged(lens, seed=len(lens)), 24, 16, seed=3)
    check(Ragged(lens, seed=len(lens), none=(1, len(lens) - 1)), 40, 8, seed=4, bf16=True, gate=False)


def test_more_sequences_than_are_looked_up_at_once():
    """1,100 single tokens, then 1,100 of up to two, in one call and in parts: the same bits."""
    import torch
    n, channels, dstate = 1100, 2048, 64
    for lens in ([1] * n, [1, 2] * (n // 2), [1, 0, 1, 2] * (n // 4)):
        r = Ragged(lens, seed=14)
        v = make(r, channels, dstate, 14, bf16=True)
        y, pool = torch.empty_like(v["x"]), v["pool"].clone()
        call(r, v, y, pool)
        z, other = torch.empty_like(y), v["pool"].clone()
        for lo in range(0, n, 220):
            rows = slice(int(r.start[lo]), int(r.start[lo + 220]))
            part = Ragged(lens[lo:lo + 220], seed=14)
            part.slots = r.slots
            part.cache_indices.copy_(r.cache_indices[lo:lo + 220])
            part.has_initial_state.copy_(r.has_initial_state[lo:lo + 220])
            call(part, {k: t[rows] if k in ("x", "dt", "B", "C", "z") else t for k, t in v.items()}, z[rows], other)
        assert same_bits(z, y) and same_bits(other, pool) and r.errors.item() == 0


@pytest.mark.parametrize("channels", [8, 56, 64, 136, 520])
@pytest.mark.parametrize("dstate", [8, 16, 32, 64])
def test_channels(channels, dstate):
    check(Ragged([45, 1, 0, 12], seed=1), channels, dstate)


@pytest.mark.parametrize("options", [dict(gate=False), dict(bf16=True), dict(D=False), dict(bias=False),
                                     dict(softplus=False), dict(softplus=False, gate=False, bf16=True)])
@pytest.mark.parametrize("dstate", [16, 32])
def test_options(options, dstate):
    check(Ragged([45, 1, 0, 12, 1], seed=2), 72, dstate, **options)


def test_strided_and_padded():
    """Column slices, rows behind the last sequence, sequences without a slot."""
    check(Ragged([40, 1, 3, 0], seed=3, rows=100, none=(1, 3)), 72, 16, strided=True)
    check(Ragged([0, 0], seed=3, rows=33), 64, 8, strided=True, gate=False)


def test_small_and_large_steps():
    """Steps down to 1e-12 keep their relative precision, those past 20 are the sum itself;
    long memories and decays that underflow."""
    import torch

    def small(v):
        v["dt_bias"][:] = torch.linspace(-27, -5, v["dt_bias"].numel())
        v["dt"] *= 0.1
        v["pool"] *= 0
    check(Ragged([200, 3], seed=4), 72, 16, change=small, gate=False)

    def large(v):
        v["dt_bias"][:] = torch.linspace(5, 60, v["dt_bias"].numel())
        v["A"][:, ::2] *= 20
        v["A"][:, 1::2] = -1e-4
    check(Ragged([50, 3], seed=5), 72, 16, change=large)


def test_infinities_and_nan():
    """They stay in their channel (x, dt, z) or token and sequence (B, C), and a gate's do
    not reach the states."""
    def change(v):
        v["x"][3, 5] = float("inf")
        v["z"][10, 6] = float("nan")
        v["z"][10, 7] = -float("inf")
        v["C"][12, 2] = float("nan")
        v["dt"][20, 9] = float("nan")
        v["pool"][:, 11, 1] = float("nan")
    check(Ragged([17, 30, 1, 0, 5], seed=6), 72, 16, change=change)


def test_parts_equal_one_prompt():
    """A prompt in parts and single tokens, through its slot."""
    import torch
    n = 75
    r = Ragged([n], seed=7)
    v = make(r, 136, 16, 7)
    y, pool = torch.empty_like(v["x"]), v["pool"].clone()
    r.has_initial_state[:] = False
    call(r, v, y, pool)
    z, other = torch.empty_like(y), v["pool"].clone()
    for lo, hi in zip([0, 1, 2, 35, 43, 74], [1, 2, 35, 43, 74, n]):
        part = Ragged([hi - lo], seed=7)
        part.has_initial_state[:] = lo > 0
        call(part, {k: t[lo:hi] if k in ("x", "dt", "B", "C", "z") else t for k, t in v.items()}, z[lo:hi], other)
    assert (f64(other) - f64(pool)).max() <= 2.0 ** -20 * np.abs(f64(pool)).max()
    d = np.abs(f64(z) - f64(y))
    assert (d <= 2 * U * np.abs(f64(y)) + 2.0 ** -18 * np.abs(f64(y)).max()).all()


def test_device_side_errors():
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    from mamba_ssd_chunked_varlen_gb300 import binding
    for offsets in ([0, 8, 4, 20], [1, 8, 9, 20], [0, 8, 9, 21], [0, -3, 9, 20]):
        r = Ragged([8, 5, 7], seed=8)
        v = make(r, 64, 16, 8)
        r.query_start_loc.copy_(torch.tensor(offsets))
        y, pool = torch.empty_like(v["x"]), v["pool"].clone()
        call(r, v, y, pool)
        assert r.errors.item() == binding.DEVERR_BAD_QUERY_START_LOC
        rest = [s for s in range(r.slots) if s not in r.slot]
        assert same_bits(pool[rest], v["pool"][rest])
    r = Ragged([8, 5, 7], seed=8)
    y, pool = torch.empty_like(v["x"]), v["pool"].clone()
    call(r, v, y, pool)
    r.cache_indices[1] = r.slots
    z, other = torch.empty_like(y), v["pool"].clone()
    call(r, v, z, other)
    assert r.errors.item() == binding.DEVERR_BAD_CACHE_INDEX
    slot = int(r.slot[1])
    assert same_bits(other[slot], v["pool"][slot])
    other[slot] = pool[slot]
    assert same_bits(other, pool) and same_bits(z[:8], y[:8]) and same_bits(z[13:], y[13:])


def test_offsets_that_fall_are_not_cut():
    """Sequences that come to far more tokens than there are rows: flagged, and nothing but
    the rows and the named slots is touched."""
    import torch
    from mamba_ssd_chunked_varlen_gb300 import binding
    n = 2000
    r = Ragged([n] + [0] * 41, seed=11)
    r.query_start_loc.copy_(torch.tensor([0, n] * 21 + [n]))
    v = make(r, 24, 16, 11)
    size = 1 << 20
    wide = torch.full((size + (1 << 16),), 77, dtype=torch.uint8, device="cuda")
    y, pool = torch.empty_like(v["x"]), v["pool"].clone()
    import mamba_ssd_chunked_varlen_gb300 as pkg
    need = pkg.ssd_selective_scan_varlen_workspace_size(n, 42, 24, 16)
    assert need <= size
    call(r, v, y, pool, workspace=wide[:need])
    assert r.errors.item() == binding.DEVERR_BAD_QUERY_START_LOC
    assert (wide[need:] == 77).all()
    rest = [s for s in range(r.slots) if s not in r.slot]
    assert same_bits(pool[rest], v["pool"][rest])


def test_workspace_is_not_overrun():
    """Cut sequences of many sizes with a workspace of exactly the size asked for."""
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    for lens, channels, dstate in (([3000], 8, 8), ([900, 3000, 40], 264, 16), ([2500], 2048, 16),
                                   ([1000] * 3, 72, 64)):
        r = Ragged(lens, seed=12)
        v = make(r, channels, dstate, 12)
        need = pkg.ssd_selective_scan_varlen_workspace_size(r.rows, len(lens), channels, dstate)
        wide = torch.full((need + (1 << 16),), 77, dtype=torch.uint8, device="cuda")
        y, pool = torch.empty_like(v["x"]), v["pool"].clone()
        call(r, v, y, pool, workspace=wide[:need])
        assert (wide[need:] == 77).all() and r.errors.item() == 0


def test_far_slots():
    """A slot past 2^31 elements, of single tokens and of a prompt that is cut."""
    import torch
    channels, dstate = 1 << 16, 16
    slots = (1 << 31) // (channels * dstate) + 3
    pool = torch.zeros(slots, channels, dstate, dtype=torch.bfloat16, device="cuda")
    for lens in ([1], [300]):
        r = Ragged(lens, seed=13)
        v = make(r, channels, dstate, 13, bf16=True)
        r.has_initial_state[:] = True
        y, small = torch.empty_like(v["x"]), v["pool"].clone()
        call(r, v, y, small)
        slot = int(r.slot[0])
        pool[-1] = v["pool"][slot]
        r.cache_indices[0] = slots - 1
        z = torch.empty_like(y)
        call(r, v, z, pool)
        assert same_bits(z, y) and same_bits(pool[-1], small[slot])
        assert not pool[:-1].any()


def test_stream_and_graph():
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    check(Ragged([37, 1, 4], seed=9), 72, 16, stream=torch.cuda.Stream())
    r = Ragged([37, 1, 4], seed=9)
    v = make(r, 72, 16, 9)
    y, pool = torch.empty_like(v["x"]), v["pool"].clone()
    workspace = pkg.alloc_selective_scan_workspace(r.rows, 3, 72, 16)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(r, v, y, pool, workspace=workspace)
    pool.copy_(v["pool"])
    for _ in range(2):
        want, kept = torch.empty_like(y), pool.clone()
        graph.replay()
        call(r, v, want, kept)
        torch.cuda.synchronize()
        assert same_bits(y, want) and same_bits(pool, kept)


def test_far_rows():
    """Rows past 2^31 elements."""
    import torch
    wide, n = 1 << 20, 2100
    r = Ragged([n], seed=10)
    v = make(r, 64, 16, 10)
    buffer = torch.zeros(n, wide, dtype=torch.bfloat16, device="cuda")
    far = dict(v)
    for i, k in enumerate(("x", "dt", "z")):
        far[k] = buffer[:, 128 * i:128 * i + 64]
        far[k].copy_(v[k])
    for i, k in enumerate(("B", "C")):
        far[k] = buffer[:, 1024 + 64 * i:1024 + 64 * i + 16]
        far[k].copy_(v[k])
    out = buffer[:, 4096:4160]
    y, pool, other = torch.empty_like(v["x"]), v["pool"].clone(), v["pool"].clone()
    call(r, v, y, pool)
    call(r, far, out, other)
    assert same_bits(out, y) and same_bits(pool, other)
