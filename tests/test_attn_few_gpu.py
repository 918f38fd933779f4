"""Attention of few rows (decoding sequences, a few proposed tokens) against its own bound: two
bf16 per weight."""
from __future__ import annotations

import numpy as np
import pytest

from attn_helpers import Batch
from attn_few_helpers import few_ref

pytestmark = pytest.mark.gpu

CASES = {
    # lens, heads, kv heads, dim, page, window: at most 16 rows a kv head and sequence
    "one": ([(1, 1), (1, 2), (1, 3), (1, 7)], 8, 4, 64, 16, 0),
    "decode": ([(1, 5), (1, 33), (1, 129), (1, 700)], 8, 2, 128, 16, 0),
    "decode_mqa": ([(1, 9), (1, 300)], 16, 1, 64, 32, 0),
    "verify": ([(5, 5), (5, 6), (5, 260), (4, 129)], 6, 2, 64, 32, 0),
    "verify_wide": ([(4, 4), (4, 9), (3, 200)], 8, 2, 128, 64, 0),
    "window": ([(5, 9), (4, 333), (1, 90)], 6, 2, 64, 16, 21),
}


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("case", CASES)
def test_two_parts_per_weight(case, kind):
    lens, heads, kv_heads, dim, page, window = CASES[case]
    b = Batch(lens, heads, kv_heads, dim, page, kind, seed=40 + len(case)).fill()
    o, _ = b.attend(window=window)
    o, q = (t.float().cpu().double().numpy() for t in (o, b.q))
    ks, vs = b.stored()
    at = 0
    for s, (n, kv) in enumerate(lens):
        want, bound = few_ref(q[at:at + n], ks[s], vs[s], n, kv, dim ** -0.5, window)
        d = np.abs(o[at:at + n] - want)
        assert np.all(d <= bound), f"{case} sequence {s}: {(d / bound).max():.2f} of the bound"
        at += n
    assert b.errors.item() == 0
