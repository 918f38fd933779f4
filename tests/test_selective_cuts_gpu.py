"""Which sequences of the selective scan are cut, and what comes of it, against the recurrence
in 64 bits (bounds of test_selective_scan_gpu.py).

A call that may cut writes at the workspace's start how many units of work there are and how
many chunks are not their sequence's last: that says whether anything was cut."""
from __future__ import annotations

import numpy as np
import pytest

from layer_helpers import Ragged, f64, near
from test_selective_scan_gpu import call, make, scan_ref

pytestmark = pytest.mark.gpu

CHUNK = 48      # tokens of the smallest chunk; sequences of two of them on are cut


def listed(workspace):
    """Units and ends of the list in the workspace."""
    import torch
    return tuple(workspace[:8].view(torch.int32).tolist())


def test_sequences_past_the_largest_power_of_two():
    """So many tokens that the smallest chunk passes 2^15: the sequence is cut all the same."""
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    total, channels, dstate = 430_000, 1536, 64
    assert total * (channels * dstate // 256) // 5000 > 1 << 15
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)

    r = Ragged([total], seed=1)
    r.has_initial_state[:] = False
    v = dict(x=normal(total, channels), dt=normal(total, channels) * 0.5, B=normal(total, dstate), C=normal(total, dstate),
             z=None, A=-(torch.rand(channels, dstate, generator=g, device="cuda") + 0.5), D=normal(channels).float(),
             dt_bias=torch.ones(channels, device="cuda"))
    y, pool = torch.empty_like(v["x"]), torch.zeros(r.slots, channels, dstate, device="cuda")
    workspace = pkg.alloc_selective_scan_workspace(total, 1, channels, dstate)
    call(r, v, y, pool, workspace=workspace)
    torch.cuda.synchronize()
    assert r.errors.item() == 0
    units, ends = listed(workspace)
    assert ends >= 3 and units == ends
    some = [0, 1, 77, 1024, channels - 1]
    cut = {k: None if t is None else t[some] if k in ("A", "D", "dt_bias") else t for k, t in v.items()}
    # its start, a place far from it and its end (600 tokens, of steps of 1.3 on average, decay by
    # exp(-390): more than fp32 holds)
    for lo, hi in ((0, 300), (total // 2 - 700, total // 2 + 100), (total - 700, total)):
        part = Ragged([hi - lo], seed=1)
        part.has[:] = False
        ref = {k: None if t is None else f64(t if k in ("A", "D", "dt_bias") else t[lo:hi, some] if k in ("x", "dt")
                                             else t[lo:hi]) for k, t in cut.items()}
        want, bound, states, off = scan_ref(part, ref, np.zeros((part.slots, len(some), dstate)), True, False)
        skip = 0 if lo == 0 else 600
        near(f64(y[lo:hi, some])[skip:], want[skip:], bound[skip:] + 2.0 ** -60, "y")
        if hi == total:
            s = int(part.slot[0])
            near(f64(pool[int(r.slot[0])][some]), states[s], off[s] + 2.0 ** -60, "pool")


def run(lens, channels, dstate, seed=0, **options):
    """Rows and slots against the recurrence; the list in the workspace."""
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    r = Ragged(lens, seed=seed)
    v = make(r, channels, dstate, seed, **options)
    y, pool = torch.empty_like(v["x"]), v["pool"].clone()
    workspace = pkg.alloc_selective_scan_workspace(r.rows, len(lens), channels, dstate)
    workspace.zero_()
    call(r, v, y, pool, workspace=workspace)
    torch.cuda.synchronize()
    ref = {k: None if t is None else f64(t) for k, t in v.items()}
    want, bound, states, off = scan_ref(r, ref, f64(v["pool"]), True, pool.dtype == torch.bfloat16)
    near(f64(y), want, bound, "y")
    near(f64(pool), states, off, "pool")
    assert r.errors.item() == 0
    return listed(workspace)


@pytest.mark.parametrize("n,ends", [(CHUNK - 1, 0), (CHUNK, 0), (CHUNK + 1, 0), (2 * CHUNK - 1, 0), (2 * CHUNK, 1),
                                    (2 * CHUNK + 1, 1), (3 * CHUNK - 1, 1), (3 * CHUNK, 2), (3 * CHUNK + 1, 2),
                                    (4 * CHUNK - 16, 2), (257, 4), (1000, 15)])
@pytest.mark.parametrize("dstate", [8, 16, 64])
def test_around_the_smallest_chunks(n, ends, dstate):
    """Chunks are n / k tokens for k = floor(n / 48), rounded up to 16: 95 tokens are none, 96 two
    of 48, 97 a chunk of 64 and one of 33, 1,000 fifteen of 64 and one of 40."""
    k = max(1, n // CHUNK)
    size = ((n + k - 1) // k + 15) // 16 * 16
    assert ends == (0 if n < 2 * CHUNK else (n + size - 1) // size - 1)
    assert run([n], 24, dstate, seed=n)[1] == ends
    run([1, n, 0, n + 1, 3, n - 1], 24, dstate, seed=n, bf16=True, gate=False)


@pytest.mark.parametrize("lens,units,ends", [
    # 14 and 10 chunks that are not the last; the sequences of few tokens are another kernel's
    ([1] * 600 + [900, 0, 2, 700] + [1] * 3, 24, 24),
    # 46 and 17 of them, and 1,043 whole sequences
    ([20] * 540 + [3000, 0, 9] + [30] * 500 + [1100, 7], 1106, 63),
])
def test_cut_sequences_behind_the_first_512(lens, units, ends):
    """The list's threads keep their first sequence's offsets, and read those of further ones again."""
    assert run(lens, 8, 16, seed=len(lens)) == (units, ends)


@pytest.mark.parametrize("channels,dstate,cut", [(6400, 16, True), (6528, 16, False), (1600, 64, True), (1664, 64, False)])
def test_wide_sequences_are_not_cut(channels, dstate, cut):
    """400 warps (of 256 states) are cut, 408 are more than two thirds of 152 SMs' schedulers: no list is
    made, also for a lone sequence."""
    assert run([400], channels, dstate, seed=channels) == ((6, 6) if cut else (0, 0))


def test_parts_equal_one_prompt_on_both_sides():
    """A prompt in parts and single tokens, through its slot: states neither larger nor smaller."""
    import torch
    n = 375
    r = Ragged([n], seed=7)
    v = make(r, 136, 16, 7)
    r.has_initial_state[:] = False
    r.has[:] = False
    y, pool = torch.empty_like(v["x"]), v["pool"].clone()
    call(r, v, y, pool)
    z, other = torch.empty_like(y), v["pool"].clone()
    for lo, hi in zip([0, 1, 2, 35, 43, 300, 374], [1, 2, 35, 43, 300, 374, n]):
        part = Ragged([hi - lo], seed=7)
        part.has_initial_state[:] = lo > 0
        call(part, {k: t[lo:hi] if k in ("x", "dt", "B", "C", "z") else t for k, t in v.items()}, z[lo:hi], other)
    ref = {k: f64(t) for k, t in v.items()}
    want, bound, states, off = scan_ref(r, ref, f64(v["pool"]), True, False)
    # each is within the bound of the recurrence
    for a, b in ((y, pool), (z, other)):
        near(f64(a), want, bound, "y")
        near(f64(b), states, off, "pool")
    slot = int(r.slot[0])
    assert np.abs(f64(other)[slot] - f64(pool)[slot]).max() <= 2 * off[slot].max()


def test_two_prompts_of_8_states_take_one_round():
    """256 CTAs with 8 states: two an SM with blocks of 16 tokens, one with those of 32.  They take less
    than 1.75 times what half of them take, one an SM (220 and 142 us: 1.55; 275, 1.94, in two rounds)."""
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    n, channels, dstate = 2000, 16384, 8

    def time_of(batch):
        r = Ragged([n] * batch, seed=1)
        g = torch.Generator(device="cuda").manual_seed(2)
        x = torch.randn(r.rows, channels, generator=g, device="cuda").bfloat16()
        B = torch.randn(r.rows, dstate, generator=g, device="cuda").bfloat16()
        A = -torch.ones(channels, dstate, device="cuda")
        y, pool = torch.empty_like(x), torch.zeros(r.slots, channels, dstate, device="cuda")
        workspace = pkg.alloc_selective_scan_workspace(r.rows, batch, channels, dstate)
        best = 1e9
        for _ in range(20):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            torch.cuda.synchronize()
            a.record()
            for _ in range(4):
                pkg.ssd_selective_scan_varlen_fwd(y, x, x, A, B, B, None, x, None, pool, *r.where, workspace=workspace)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b) / 4)
        return best
    assert time_of(2) < 1.75 * time_of(1)
