"""The selective scan of batches that are mostly empty sequences, as a captured step of a fixed
size is, with long sequences among them."""
from __future__ import annotations

import pytest

from layer_helpers import Ragged
from test_selective_scan_gpu import check

pytestmark = pytest.mark.gpu

LENS = [
    [0] * 10 + [9] + [0] * 3, [10] + [0] * 9, [0] * 20 + [17, 0, 1] + [0] * 9, [0] * 200 + [9, 60, 0, 25, 100, 0, 1, 2, 3],
    [1] * 20 + [0] * 90 + [41] + [0] * 30 + [33, 16, 24] + [1] * 7,
]


@pytest.mark.parametrize("lens", range(len(LENS)))
@pytest.mark.parametrize("dstate", [8, 16, 32, 64])
def test_long_ones_among_empty_ones(lens, dstate):
    lens = LENS[lens]
    assert sum(lens) <= len(lens)
    check(Ragged(lens, seed=len(lens)), 72, dstate, seed=dstate)
    check(Ragged(lens, seed=len(lens), rows=sum(lens), none=(len(lens) // 3,)), 264, dstate, bf16=True, gate=False)


@pytest.mark.parametrize("lens", [[9] * 10 + [0] * 80, [0] * 3 + [9] * 30 + [8] * 10 + [0] * 2, [9, 0] * 40 + [100] + [0] * 90])
@pytest.mark.parametrize("channels,dstate", [(2056, 8), (1032, 16), (264, 64)])
def test_as_many_long_ones_as_there_can_be(lens, channels, dstate):
    """Sequences of nine tokens are the shortest that the kernel of few tokens leaves to the other."""
    check(Ragged(lens, seed=len(lens)), channels, dstate, seed=dstate)


@pytest.mark.parametrize("dstate", [8, 16, 32, 64])
def test_strided_and_padded(dstate):
    check(Ragged([0] * 70 + [30, 12], seed=3, rows=60), 72, dstate, strided=True)
    check(Ragged([0] * 70 + [30, 12], seed=3, rows=60), 8, dstate, softplus=False, D=False, bias=False)


def test_a_prompt_costs_no_more_than_a_few_times_itself():
    """Its tokens are on their way while earlier ones are worked on: 500 of them take up to 6 times
    what they take without the empty sequences (cut into chunks there), not 20 times."""
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    n, channels, dstate = 500, 2048, 16

    def time_of(lens):
        x = torch.randn(n, channels, device="cuda").bfloat16()
        B = torch.randn(n, dstate, device="cuda").bfloat16()
        A = -torch.ones(channels, dstate, device="cuda")
        y, pool = torch.empty_like(x), torch.zeros(len(lens), channels, dstate, device="cuda")
        start = torch.zeros(len(lens) + 1, dtype=torch.int32)
        start[1:] = torch.tensor(lens).cumsum(0)
        start, slots = start.cuda(), torch.arange(len(lens), dtype=torch.int32, device="cuda")
        workspace = pkg.alloc_selective_scan_workspace(n, len(lens), channels, dstate)
        best = 1e9
        for _ in range(20):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            torch.cuda.synchronize()
            a.record()
            for _ in range(10):
                pkg.ssd_selective_scan_varlen_fwd(y, x, x, A, B, B, None, None, None, pool, start, None, slots,
                                                  workspace=workspace)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b) / 10)
        return best
    assert time_of([0] * 250 + [n] + [0] * 261) < 6 * time_of([n])
