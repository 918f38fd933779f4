"""Host-side checks of ssd_scan_varlen_fwd_strided's views (no GPU)."""
from __future__ import annotations

import pytest
import torch

from mamba_ssd_chunked_varlen_gb300 import binding


class OnDevice(torch.Tensor):
    """A CPU tensor that says it is on the device: for checks that come before any launch."""

    is_cuda = property(lambda self: True)


def view(t):
    return t.as_subclass(OnDevice)


def test_expanded_views_are_refused():
    """An expanded view has a token stride of 0, which the C ABI takes as contiguous: the
    call would read, or write, rows past the view's end."""
    row = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    half = torch.zeros(5 * 128, dtype=torch.bfloat16).as_strided((5, 2, 64), (64, 64, 1))
    for t in (row.expand(5, 2, 64), half):
        with pytest.raises(ValueError, match="overlap"):
            binding._token_major(view(t), "x", torch.bfloat16, 128)
    with pytest.raises(ValueError, match="overlap"):
        binding._token_major(view(torch.zeros(1, 4, dtype=torch.bfloat16).expand(5, 4)), "dt",
                             torch.bfloat16, 4)


def test_wide_and_single_rows_pass():
    wide = torch.zeros(5, 300, dtype=torch.bfloat16)[:, 8:136].view(5, 2, 64)
    assert binding._token_major(view(wide), "x", torch.bfloat16, 128)[1] == 300
    one = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    assert binding._token_major(view(one), "x", torch.bfloat16, 128)[1] == 128
    assert binding._token_major(view(one.as_strided((1, 2, 64), (0, 64, 1))), "x", torch.bfloat16, 128)[1] == 0
