"""Edges of the attention over the paged cache, on the GPU, against the 64-bit
answer with the bounds that attn_helpers derives (or its own, where stated)."""
from __future__ import annotations

import numpy as np
import pytest

from attn_helpers import Batch, check_attend

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "fp8", "int8"]


def padded(lens, kv, *args, **kw):
    """A batch of `lens` whose kv_lens are then set to `kv`: rows at negative positions."""
    import torch
    b = Batch(lens, *args, **kw).fill()
    b.kv_lens.copy_(torch.tensor(kv))
    b.lens = [(n, k) for (n, _), k in zip(lens, kv)]
    return b


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 64, 2 ** 30, 2 ** 30 - 1])
def test_window_of_no_limit(kind, window):
    """A window wider than any context is none, beside padding rows as well (their
    positions are negative: less a window of 2^31 they leave 32 bits)."""
    import torch
    lens, kv = [(6, 6), (130, 130), (40, 40), (1, 1)], [2, 3, 33, 1]
    b = padded(lens, kv, 4, 2, 64, 16, kind, seed=21)
    o, lse = b.attend(window=0)
    check_attend(b, o, lse, what="padding")
    o2, lse2 = b.attend(window=window)
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and b.errors.item() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [1, 3, 40])
def test_window_and_padding(kind, window):
    b = padded([(6, 6), (130, 130), (40, 60), (3, 1)], [4, 70, 60, 1], 4, 2, 64, 16, kind, seed=22)
    o, lse = b.attend(window=window)
    check_attend(b, o, lse, window=window, what="padding")


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_calls_in_a_row_have_plans_of_their_own(kind):
    """Batches of both kinds of unit in turn, in one workspace and without a stop between: each
    call's kernels go by its own plan, also where they start ahead of their predecessor's
    end."""
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    made = []
    for seed, lens in enumerate([[(1, 900), (90, 300), (1, 33)] * 4, [(70, 70), (1, 2000), (130, 131)],
                                 [(1, 50)] * 60 + [(33, 700)], [(1, 5)], [(40, 40)]]):
        b = Batch(lens, 4, 2, 64, 16, kind, seed=30 + seed).fill()
        o, lse = b.attend()
        check_attend(b, o, lse, what=f"batch {seed}")
        made.append((b, o, lse, torch.empty_like(o), torch.empty_like(lse)))
    ws = pkg.alloc_attn_workspace(max(b.total for b, *_ in made), 64, 4, 2, 64)
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(20):
        for b, o, lse, o2, lse2 in made:
            pkg.ssd_attn_varlen_fwd(o2, lse2, b.q, *b.cache, *b.where, softmax_scale=0.125,
                                    workspace=ws, errors=b.errors)
        for b, o, lse, o2, lse2 in made:
            wrong += (o != o2).sum() + (lse != lse2).sum()
            o2.zero_()
            lse2.zero_()
    assert wrong.item() == 0 and all(b.errors.item() == 0 for b, *_ in made)


def spoil(b, what):
    """Keys that rows of the batch do not see, and some that they do, get a factor of zero, or
    a negative one: what `stored` then gives for them is what the definition says."""
    import torch
    ks, vs = None, None
    if what == "bad page":
        b.block_table[0, 3] = -1
        b.block_table[0, 18] = 1 << 20
        ks, vs = b.stored()
        for x in (ks[0], vs[0]):
            x[48:64] = 0.0
            x[288:300] = 0.0
        return ks, vs
    for j in (5, 60, 283, 290, 299):
        p, r = b.row_of(0, j)
        b.k_scale[p, :, r] *= 0.0 if what == "zero scale" else -1.0
    return b.stored()


@pytest.mark.parametrize("softmax_scale", [None, -0.1])
@pytest.mark.parametrize("new", [3, 20])
@pytest.mark.parametrize("what", ["bad page", "zero scale", "negative scale"])
@pytest.mark.parametrize("kind", ["fp8", "int8"])
def test_hidden_keys_of_any_factor(kind, what, new, softmax_scale):
    """A key whose scale is zero or negative, or whose page is out of range (it reads as zeros),
    is hidden from the rows before it like any other."""
    from mamba_ssd_chunked_varlen_gb300 import attention
    b = Batch([(new, 300), (1, 90)], 4, 2, 64, 16, kind, seed=23).fill()
    stored = spoil(b, what)
    o, lse = b.attend(softmax_scale=softmax_scale)
    check_attend(b, o, lse, softmax_scale=softmax_scale, what=what, stored=stored)
    assert b.errors.item() == (attention.DEVERR_BAD_PAGE if what == "bad page" else 0)


@pytest.mark.parametrize("new", [2, 40])
@pytest.mark.parametrize("kind", ["fp8", "int8"])
@pytest.mark.parametrize("softmax_scale", [0.0, 1e-30, -0.1])
def test_softmax_scale_of_quantised_cache(softmax_scale, kind, new):
    """A softmax_scale of zero gives means also where the product with a key's scale is below
    fp32's numbers: small keys, and rows of zeros."""
    b = Batch([(new, 300), (20, 20)], 4, 2, 64, 16, kind, seed=24)
    for k in b.k_seq:
        k[::3] *= 2.0 ** -50
        k[1::7] = 0.0
    b.fill()
    o, lse = b.attend(softmax_scale=softmax_scale)
    check_attend(b, o, lse, softmax_scale=softmax_scale, what="scale")


@pytest.mark.parametrize("kv,new,dim,window",
                         [(kv, new, dim, window) for kv in (310, 5000) for new in (1, 4, 6, 8, 40)
                          for dim in (64, 128) for window in (0, 290)]
                         + [(120001, new, dim, 0) for new in (1, 6) for dim in (64, 128)])
def test_infinite_values(kv, new, dim, window):
    """An infinity in V is the result of every row that sees it, with its sign, in the keys'
    first tiles as in the last; so is NaN, and so is NaN where both infinities meet.  The
    other columns, and the rows that do not see it, are as they were."""
    import torch
    # (a second sequence, so that the first is cut in several ways)
    b = Batch([(new, kv), (1, 64)], 4, 2, dim, 16, "bf16", seed=25).fill()
    clean, clean_lse = b.attend(window=window)
    inf = float("inf")
    keys = [kv - 289, kv - 200, kv - 2 if new > 1 else kv - 1]
    for j, (up, down) in zip(keys, ((3, 9), (17, 30), (40, 57))):
        p, r = b.row_of(0, j)
        b.v_cache[p, 0, r, up] = inf
        b.v_cache[p, 0, r, down] = -inf
        b.v_cache[p, 1, r, up] = float("nan")
        b.v_cache[p, 0, r, 60] = inf
        p, r = b.row_of(0, j - 5)
        b.v_cache[p, 0, r, 61] = -inf
        b.v_cache[p, 1, r, 62] = inf
        b.v_cache[p, 1, r, 63] = -inf
    p, r = b.row_of(0, kv - 250)
    b.v_cache[p, 1, r, 62] = -inf
    o, lse = b.attend(window=window)
    # by the definition, column by column: sums of what a row sees
    _, vs = b.stored()
    want = clean.float().cpu().numpy()
    for i in range(new):
        at = kv - new + i
        lo = max(0, at - window + 1) if window else 0
        with np.errstate(invalid="ignore"):      # (both infinities)
            seen = np.where(np.isfinite(vs[0]), 0.0, vs[0])[lo:at + 1].sum(0)  # (kv heads, dim)
        for h in range(4):
            want[i, h] = np.where(seen[h // 2] == 0, want[i, h], seen[h // 2])
    assert np.array_equal(o.float().cpu().numpy(), want, equal_nan=True)
    assert torch.equal(lse, clean_lse)


@pytest.mark.parametrize("case", ["few", "few16", "tiles", "wide"])
@pytest.mark.parametrize("kind", KINDS)
def test_values_of_a_negligible_piece(kind, case):
    """NaN (bf16: and infinities) in V reach the rows that see them also where all keys of the
    piece that they lie in have probabilities of 2^-738, and no column or row but theirs."""
    import torch
    new, kv, lo, hi, at = {"few": (1, 400, 32, 64, 40), "few16": (5, 400, 32, 64, 40),
                           "tiles": (40, 700, 128, 256, 200), "wide": (1, 70000, 32000, 32320, 32160)}[case]
    b = Batch([(new, kv)], 4, 2, 64, 16, kind, seed=26) if case != "wide" else \
        Batch([(new, kv)], 2, 1, 64, 16, kind, seed=26)
    b.q.fill_(8.0)
    b.k_seq[0].mul_(0.125)
    b.k_seq[0][lo:hi] = -8.0
    b.fill()
    clean, clean_lse = b.attend()
    p, r = b.row_of(0, at)
    if kind == "bf16":
        b.v_cache[p, 0, r, 7] = float("nan")
        b.v_cache[p, 0, r, 8] = float("inf")
        b.v_cache[p, 0, r, 9] = -float("inf")
    else:
        b.v_scale[p, 0, r] = float("nan")
    o, lse = b.attend()
    if kind == "bf16":
        assert torch.isnan(o[:, :2, 7]).all()
        assert (o[:, :2, 8] == float("inf")).all() and (o[:, :2, 9] == -float("inf")).all()
        o[:, :2, 7:10] = clean[:, :2, 7:10]
    else:
        assert torch.isnan(o[:, :2]).all()
        o[:, :2] = clean[:, :2]
    assert torch.equal(o, clean) and (kind != "bf16" or torch.equal(lse, clean_lse))


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_more_sequences_than_the_plan_keeps_on_chip(kind):
    """Over 4,096 sequences, of both kinds of unit, and more units of a kind than 1,024."""
    lens = [(1, 1 + 5 * b % 60) for b in range(4300)] + [(20, 30), (0, 9), (3, 3)] * 20 + [(9, 140)]
    b = Batch(lens, 2, 1, 64, 16, kind, seed=27).fill()
    o, lse = b.attend()
    check_attend(b, o, lse, what="many")
    assert b.errors.item() == 0


@pytest.mark.parametrize("kind,window", [("bf16", 0), ("int8", 0), ("fp8", 100)])
def test_far_pages(kind, window):
    """Pages past 2^31 elements into the cache."""
    b = Batch([(1, 700), (40, 300), (5, 90)], 4, 2, 64, 256, kind, seed=28)
    page = 256 * 2 * 64
    b.pages = (1 << 31) // page + 8
    near = b.table_cpu < 1 << 30
    b.table_cpu = b.table_cpu.where(~near, b.pages - 1 - b.table_cpu)
    b.block_table.copy_(b.table_cpu)
    b.k_cache = b.k_cache.new_zeros((b.pages, 2, 256, 64))
    b.v_cache = b.k_cache.clone()
    if kind != "bf16":
        b.k_scale = b.k_scale.new_zeros((b.pages, 2, 256))
        b.v_scale = b.k_scale.clone()
    b.fill()
    o, lse = b.attend(window=window)
    # (the pages in use alone, counted from the first of them)
    low = b.pages - 8 - 1
    for name in ("k_cache", "v_cache", "k_scale", "v_scale"):
        if getattr(b, name) is not None:
            setattr(b, name, getattr(b, name)[low:].clone())
    b.table_cpu = b.table_cpu.where(~near, b.table_cpu - low)
    check_attend(b, o, lse, window=window, what="far")
    assert b.errors.item() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_large_values(kind):
    """Values of 2^79 while the scores grow from key to key, so that the reference lags behind
    the maximum: the sums stay finite."""
    import torch
    b = Batch([(1, 900), (5, 500), (60, 700)], 4, 2, 64, 32, kind, seed=29)
    for k, v in zip(b.k_seq, b.v_seq):
        k.abs_().mul_(torch.linspace(0.0, 1.5, k.shape[0])[:, None, None]).copy_(k)
        v.sign_().mul_(2.0 ** 79)
    b.q.abs_()
    b.fill()
    o, lse = b.attend()
    check_attend(b, o, lse, what="large")


@pytest.mark.parametrize("kind", KINDS)
def test_tiles_without_a_page(kind):
    """Whole key tiles whose pages are out of range read as zeros, one after the other and between
    tiles that are there."""
    from mamba_ssd_chunked_varlen_gb300 import attention
    b = Batch([(40, 1500), (2, 600)], 4, 2, 64, 32, kind, seed=33).fill()
    ks, vs = b.stored()
    for seq, lo, hi in ((0, 128, 640), (0, 768, 896), (0, 1024, 1280), (1, 0, 256)):
        b.block_table[seq, lo // 32:hi // 32] = b.pages
        ks[seq][lo:hi] = 0.0
        vs[seq][lo:hi] = 0.0
    for _ in range(5):
        o, lse = b.attend()
        check_attend(b, o, lse, what="no page", stored=(ks, vs))
    assert b.errors.item() == attention.DEVERR_BAD_PAGE
