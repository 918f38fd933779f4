"""Attention of new tokens over the paged cache, on the GPU, against the 64-bit
answer with the bounds that attn_helpers derives."""
from __future__ import annotations

import numpy as np
import pytest

from attn_helpers import Batch, check_attend

pytestmark = pytest.mark.gpu

CASES = {
    # lens, heads, kv heads, dim, page, window
    "one": ([(1, 1)], 1, 1, 64, 16, 0),
    "decode": ([(1, 1), (1, 2), (1, 127), (1, 128), (1, 129), (1, 700)], 8, 2, 128, 16, 0),
    "decode_mqa": ([(1, 300), (1, 16)], 16, 1, 64, 32, 0),
    "group_of_128": ([(1, 40), (3, 150)], 128, 1, 64, 16, 0),
    "group_of_100": ([(2, 140)], 100, 1, 128, 32, 0),
    "verify": ([(5, 5), (5, 6), (5, 260), (4, 129), (5, 1001)], 6, 2, 64, 32, 0),
    "odd_groups": ([(70, 333), (1, 90), (0, 50), (23, 23)], 14, 2, 128, 64, 0),
    "prompt": ([(257, 257), (128, 128), (129, 129), (1, 1)], 2, 2, 64, 128, 0),
    "chunk": ([(200, 900)], 4, 1, 128, 256, 0),
    "chunk_g3": ([(100, 513), (31, 777)], 3, 1, 128, 16, 0),
    "window": ([(150, 400), (1, 333), (64, 64), (5, 1000)], 4, 2, 64, 16, 50),
    "window_1": ([(40, 300), (1, 129)], 2, 1, 128, 32, 1),
    "window_129": ([(140, 600), (1, 259)], 2, 2, 64, 64, 129),
    "window_wide": ([(20, 100)], 2, 1, 64, 16, 5000),
    "empty_among": ([(0, 0), (3, 9), (0, 40), (0, 0), (1, 5)], 4, 4, 64, 16, 0),
}


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("case", CASES)
def test_attend(case, kind):
    lens, heads, kv_heads, dim, page, window = CASES[case]
    b = Batch(lens, heads, kv_heads, dim, page, kind, seed=len(case)).fill()
    o, lse = b.attend(window=window)
    check_attend(b, o, lse, window=window, what=case)
    assert b.errors.item() == 0


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_sharp_rows(kind):
    """Scores of hundreds: the running maximum moves far from tile to tile, in
    both directions, and some rows are all on one key."""
    import torch
    b = Batch([(3, 900), (130, 700)], 4, 2, 64, 32, kind, seed=3, q_scale=6.0)
    for k in b.k_seq:
        k.mul_(torch.linspace(0.2, 4.0, k.shape[0])[:, None, None]).copy_(k)
    b.k_seq[1] = b.k_seq[1].flip(0).contiguous()
    b.fill()
    o, lse = b.attend(softmax_scale=0.5)
    check_attend(b, o, lse, softmax_scale=0.5, what="sharp")


@pytest.mark.parametrize("scale", [0.0, -0.1])
def test_softmax_scale(scale):
    """A scale of zero gives means, a negative one is taken as it is."""
    b = Batch([(2, 300), (20, 20)], 4, 2, 64, 16, "bf16", seed=4).fill()
    o, lse = b.attend(softmax_scale=scale)
    check_attend(b, o, lse, softmax_scale=scale, what="scale")


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_value_scales_apart(kind):
    """Values of very different sizes from token to token, zero rows among them:
    the zero rows count in the sum of the probabilities."""
    import torch
    b = Batch([(1, 400), (40, 290)], 2, 1, 64, 16, kind, seed=9)
    for v in b.v_seq:
        n = v.shape[0]
        v.mul_(torch.exp2(torch.randint(-40, 20, (n, 1, 1)).float())).copy_(v)
        v[::3] = 0.0
        v[0] = 0.0
    for k, s in zip(b.k_seq, range(2)):
        k[0] *= 3.0
    b.fill()
    o, lse = b.attend()
    check_attend(b, o, lse, what="values")


def test_no_lse_and_same_bits():
    """Without lse, twice, and with the sequences in another order: the same bits
    of o for the same call, the same values within the bounds otherwise."""
    import torch
    lens = [(1, 1500), (60, 300), (1, 40)]
    b = Batch(lens, 8, 2, 128, 16, "bf16", seed=11).fill()
    o, lse = b.attend()
    o2, none = b.attend(lse=False)
    o3, lse3 = b.attend()
    assert none is None and torch.equal(o, o2) and torch.equal(o, o3) and torch.equal(lse, lse3)


def test_padding_rows():
    """kv_lens below the new rows: rows at negative positions see no key."""
    import torch
    b = Batch([(6, 6), (130, 130), (1, 1)], 4, 2, 64, 16, "bf16", seed=12).fill()
    b.kv_lens.copy_(torch.tensor([2, 3, 0]))
    b.k_seq = b.v_seq = None
    b.lens = [(6, 2), (130, 3), (1, 0)]
    o, lse = b.attend()
    check_attend(b, o, lse, what="padding")
    assert (o[:4] == 0).all() and torch.isinf(lse[:4]).all() and (o[6:133] == 0).all()
    assert (o[136] == 0).all() and b.errors.item() == 0


@pytest.mark.parametrize("dim,window", [(64, 0), (128, 0), (64, 20)])
def test_hidden_values_do_not_matter(dim, window):
    """Infinities and NaN in keys and values that a row's mask hides do not
    reach it; a row that sees one has it."""
    import torch
    lens = [(150, 290), (1, 200)]
    b = Batch(lens, 4, 2, dim, 16, "bf16", seed=13).fill()
    clean, clean_lse = b.attend(window=window)
    j = 260
    p, r = b.row_of(0, j)
    b.k_cache[p, 0, r] = float("nan")
    b.v_cache[p, 0, r, 5] = float("inf")
    b.v_cache[p, 1, r, 7] = float("nan")
    b.v_cache[p, 1, r, 9] = -float("inf")
    o, lse = b.attend(window=window)
    at = np.arange(150) + 140
    sees = (at >= j) & ((at < j + window) if window else True)
    sees = torch.from_numpy(np.concatenate([sees, [False]])).to(o.device)
    assert torch.equal(o[~sees], clean[~sees]) and torch.equal(lse[~sees], clean_lse[~sees])
    assert torch.isnan(o[sees][:, :2]).all() and torch.isnan(lse[sees][:, :2]).all()
    seen = o[sees][:, 2:]
    assert torch.isnan(seen[..., 7]).all() and (seen[..., 9] == -float("inf")).all()
    others = [d for d in range(dim) if d not in (7, 9)]
    torch.testing.assert_close(seen[..., others].float(), clean[sees][:, 2:][..., others].float(),
                               rtol=2 ** -7, atol=2 ** -9)


@pytest.mark.parametrize("kind", ["fp8", "int8"])
def test_hidden_rows_of_quantised_cache(kind):
    """A non-finite row of an 8-bit cache (scale NaN) reaches the rows that see
    it and no other."""
    import torch
    lens = [(150, 290), (3, 200)]
    b = Batch(lens, 4, 2, 64, 16, kind, seed=14).fill()
    clean, _ = b.attend()
    for name in ("k_scale", "v_scale"):
        b.fill()
        p, r = b.row_of(0, 260)
        getattr(b, name)[p, 1, r] = float("nan")
        o, lse = b.attend()
        sees = torch.cat([torch.arange(150) + 140 >= 260, torch.zeros(3, dtype=torch.bool)]).to(o.device)
        assert torch.equal(o[~sees], clean[~sees]) and torch.equal(o[:, :2], clean[:, :2])
        assert torch.isnan(o[sees][:, 2:]).all()


@pytest.mark.parametrize("new", [2, 40])
@pytest.mark.parametrize("kind", ["fp8", "int8"])
def test_nan_scale_of_negligible_key(kind, new):
    """A value's scale of NaN reaches the rows that see it even where the key's
    probability underflows to zero, in a tile that hides other keys."""
    import torch
    b = Batch([(new, 40)], 4, 2, 64, 16, kind, seed=11)
    b.q.fill_(8.0)
    b.k_seq[0].mul_(0.125)
    b.k_seq[0][33] = -8.0            # its score is -512: 2^-738 next to the others
    b.fill()
    p, r = b.row_of(0, 33)
    b.v_scale[p, 0, r] = float("nan")
    o, _ = b.attend()
    sees = torch.arange(40 - new, 40, device=o.device) >= 33
    assert torch.isnan(o[sees][:, :2]).all()
    assert torch.isfinite(o[~sees]).all() and torch.isfinite(o[:, 2:]).all()


def test_strides():
    """q as a slice of a fused projection, o a slice of a wider buffer, the table
    a slice of a wider one."""
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    b = Batch([(9, 140), (40, 40)], 4, 2, 64, 16, "bf16", seed=15).fill()
    o, lse = b.attend()
    wide = torch.randn(b.total, 4 * 64 * 2 + 24, device="cuda").bfloat16()
    q = wide[:, 8:264].view(b.total, 4, 64)
    q.copy_(b.q)
    out = torch.full((b.total, 4 * 64 + 16), 5.0, dtype=torch.bfloat16, device="cuda")
    o2 = out[:, 8:264].view(b.total, 4, 64)
    table = torch.full((2, b.block_table.shape[1] + 5), -7, dtype=torch.int32, device="cuda")
    table[:, 3:-2] = b.block_table
    ws = pkg.alloc_attn_workspace(b.total, 2, 4, 2, 64)
    lse2 = torch.empty_like(lse)
    pkg.ssd_attn_varlen_fwd(o2, lse2, q, *b.cache, b.query_start_loc, b.kv_lens, table[:, 3:-2],
                            softmax_scale=0.125, workspace=ws)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert (out[:, :8] == 5).all() and (out[:, 264:] == 5).all()


def test_another_stream_and_graph():
    """On a side stream, and replayed from a CUDA graph after kv_lens grew (the
    lengths are read on the device)."""
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    b = Batch([(1, 700), (1, 40)], 8, 2, 128, 16, "int8", seed=16).fill()
    o, _ = b.attend()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, _ = b.attend(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, o2)
    ws = pkg.alloc_attn_workspace(b.total, 2, 8, 2, 128)
    out = torch.empty_like(o)
    b.kv_lens.copy_(torch.tensor([5, 6]))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.ssd_attn_varlen_fwd(out, None, b.q, *b.cache, *b.where, softmax_scale=128 ** -0.5,
                                workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(out, o)
    b.kv_lens.copy_(torch.tensor([700, 40]))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, o)


def test_device_side_errors():
    import torch
    from mamba_ssd_chunked_varlen_gb300 import attention

    def make():
        return Batch([(20, 300), (1, 90)], 4, 2, 64, 16, "bf16", seed=17).fill()

    b = make()
    clean, _ = b.attend()
    # a page out of range: its keys and values are zeros
    for bad in (-1, 1 << 20):
        b = make()
        b.block_table[0, 3] = bad
        o, lse = b.attend()
        assert b.errors.item() == attention.DEVERR_BAD_PAGE
        assert torch.equal(o[20], clean[20])
        ks, vs = b.stored()
        for x in (ks[0], vs[0]):
            x[48:64] = 0.0
        check_attend(b, o, lse, what="bad page", stored=(ks, vs))
    for n in (-1, 100000):
        b = make()
        b.kv_lens[1] = n
        o, lse = b.attend()
        assert b.errors.item() == attention.DEVERR_BAD_KV_LEN
        assert (o[20] == 0).all() and torch.isinf(lse[20]).all() and torch.equal(o[:20], clean[:20])


def test_bad_query_start_loc():
    """Nothing is computed or written, the flag is set."""
    import torch
    from mamba_ssd_chunked_varlen_gb300 import binding
    for q in ([0, 20, 20], [1, 20, 21], [0, 25, 21], [0, 20, 40]):
        b = Batch([(20, 300), (1, 90)], 4, 2, 64, 16, "bf16", seed=17).fill()
        b.query_start_loc.copy_(torch.tensor(q))
        o, lse = b.attend()
        assert b.errors.item() == binding.DEVERR_BAD_QUERY_START_LOC
        assert torch.isnan(o).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_many_sequences(kind):
    """More sequences than one CTA has threads, most of one token."""
    lens = [(1, 1 + 7 * b % 200) for b in range(1500)] + [(3, 40), (0, 7), (2, 2)]
    b = Batch(lens, 2, 1, 64, 16, kind, seed=18).fill()
    o, lse = b.attend()
    check_attend(b, o, lse, what="many")


def test_long_context():
    """One token over 70,001 keys and a chunk of 33 over 20,000: the keys are
    split over many CTAs and joined."""
    b = Batch([(1, 70001), (33, 20000)], 4, 2, 64, 64, "int8", seed=19).fill()
    o, lse = b.attend()
    check_attend(b, o, lse, what="long")
