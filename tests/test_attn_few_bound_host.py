"""The bound of few rows tells two bf16 per weight from one, in short contexts (in long ones
the roundings of the weights average out below any worst case).  No GPU."""
from __future__ import annotations

import numpy as np
import pytest

from attn_few_helpers import bf16, few_model, few_ref


@pytest.mark.parametrize("n,kv", [(1, 5), (5, 9)])
def test_one_part_per_weight_is_outside(n, kv):
    rng = np.random.default_rng(n * 100 + kv)

    def draw(*shape):
        return bf16(rng.standard_normal(shape, dtype=np.float32)).astype(np.float64)

    outside = 0
    for _ in range(20):
        q, k, v = draw(n, 8, 64), draw(kv, 4, 64), draw(kv, 4, 64)
        o, bound = few_ref(q, k, v, n, kv, 0.125, 0)
        assert np.all(np.abs(few_model(q, k, v, n, kv, 0.125, 2) - o) <= bound)
        outside += int((np.abs(few_model(q, k, v, n, kv, 0.125, 1) - o) > bound).sum())
    assert outside > 0


def test_bf16_rounds_to_nearest_even():
    import torch
    x = np.random.default_rng(1).standard_normal(1000).astype(np.float32) * 2.0 ** np.arange(-100, 100).repeat(5)
    x = x.astype(np.float32)
    assert np.array_equal(bf16(x), torch.from_numpy(x).bfloat16().float().numpy())
