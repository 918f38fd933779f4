"""Which sequences of the selective scan are cut, and what comes of it, against the recurrence
in 64 bits (bounds of test_selective_scan_gpu.py).

A call that may cut writes at the workspace's start how many units of work there are and how
many chunks are not their sequence's last: that says whether anything was cut."""
from __future__ import annotations

import numpy as np
import pytest

from layer_helpers import Ragged, f64, near
from test_selective_scan_gpu import call, scan_ref

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
    total, channels, dstate = 326_000, 2048, 64
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
