"""Shared helpers of the layer operators' tests: a ragged batch with its slots."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -8        # half a step of bf16, relative
E = 2.0 ** -24       # half a step of fp32, relative


class Ragged:
    """Sequences of the given lengths in `rows` rows (0: exactly theirs), with a slot each
    (-1: none) of a pool of `slots`, half of them with an initial state."""

    def __init__(self, lens, seed=0, rows=0, none=(), device="cuda"):
        import torch
        rng = np.random.default_rng([seed, len(lens)])
        self.lens, batch = list(lens), len(lens)
        self.start = np.zeros(batch + 1, np.int64)
        self.start[1:] = np.cumsum(lens)
        self.rows = rows or int(self.start[-1])
        self.slots = batch + 3
        self.slot = rng.permutation(self.slots)[:batch]
        for b in none:
            self.slot[b] = -1
        self.has = rng.random(batch) < 0.5
        self.query_start_loc = torch.tensor(self.start, dtype=torch.int32, device=device)
        self.cache_indices = torch.tensor(self.slot, dtype=torch.int32, device=device)
        self.has_initial_state = torch.tensor(self.has, device=device)
        self.errors = torch.zeros(1, dtype=torch.int32, device=device)

    @property
    def where(self):
        return self.query_start_loc, self.has_initial_state, self.cache_indices

    def each(self):
        """(sequence, first row, end, slot or -1, whether it has an initial state)."""
        for b in range(len(self.lens)):
            yield b, int(self.start[b]), int(self.start[b + 1]), int(self.slot[b]), \
                bool(self.has[b]) and self.slot[b] >= 0


def f64(t):
    return t.detach().float().cpu().double().numpy()


def sliced(t, extra=16):
    """The same rows as a column slice of a wider buffer of NaN."""
    import torch
    wide = torch.full((t.shape[0], t[0].numel() + 2 * extra), float("nan"), dtype=t.dtype, device=t.device)
    view = wide[:, extra:extra + t[0].numel()].view(t.shape)
    view.copy_(t)
    return wide, view


def same_bits(x, y):
    import torch
    return torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))


def near(got, want, bound, what=""):
    """|got - want| <= bound where `want` is finite; NaN and infinities the same."""
    odd = ~np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN elsewhere"
    assert np.array_equal(got[odd & ~np.isnan(want)], want[odd & ~np.isnan(want)]), f"{what}: infinities"
    d = np.abs(np.where(odd, 0, got) - np.where(odd, 0, want))
    bad = ~odd & ~(d <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, off by {d.max():.3e}, " \
        f"{np.max(np.where(odd, 0, d / np.maximum(bound, 1e-300))):.2f} of the bound"
