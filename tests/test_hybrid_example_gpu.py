"""The hybrid serving example: every step's attention against the plain formula in
64 bits over the contexts that the cache gives back.

Bound, per output element, with V the largest |v| of the context.  A read-back
key is one bf16 rounding (2^-8 relative, 8-bit caches only) away from the cache's,
so a score is off by e = 2^-8 scale sum |q k| at most, and the row's weights by
factors within exp(+-2e), which moves a mean of values by at most expm1(2e) V.  The
read-back value adds 2^-8 V.  Inside the kernel a probability is rounded to bf16
once (2^-8 V), the scores and sums are fp32 (some 2^-16 V), and the output is
rounded to bf16 (2^-8 V).
"""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["bfloat16", "float8_e4m3fn", "int8"])
def test_serving_steps(cache):
    import hybrid_serving as E
    import mamba_ssd_chunked_varlen_gb300 as ssd
    block = E.HybridBlock(cache=getattr(torch, cache))
    scale, group = E.DIM ** -0.5, E.HEADS // E.KV_HEADS
    for batch, out in E.serve(block, 8):
        q, o = (t.double() for t in block.last)
        k, v, first = block.contexts()
        first, row = first.tolist(), 0
        for b, (_, n) in enumerate(batch):
            kk, vv = (t[first[b]:first[b + 1]].double().repeat_interleave(group, 1) for t in (k, v))
            qq, got = q[row:row + n], o[row:row + n]
            row += n
            keys = kk.shape[0]
            hidden = torch.arange(keys, device=q.device) > torch.arange(keys - n, keys, device=q.device)[:, None]
            x = torch.einsum("nhd,khd->nhk", qq, kk) * scale
            x = x.masked_fill(hidden[:, None], float("-inf"))
            want = torch.einsum("nhk,khd->nhd", x.softmax(-1), vv)
            e = torch.einsum("nhd,khd->nhk", qq.abs(), kk.abs()).masked_fill(hidden[:, None], 0).amax(-1)
            e = e * scale * (2.0 ** -8 if cache != "bfloat16" else 0.0)
            top = vv.abs().amax((0, 2))[None, :]
            bound = (torch.expm1(2 * e) + 3 * 2.0 ** -8 + 2.0 ** -16) * top
            assert ((got - want).abs() <= bound[..., None]).all()
        assert torch.isfinite(out).all()
    assert int(block.errors) == 0 and ssd.ssd_scan_varlen_read_errors(block.scan_ws) == 0
