"""The paged cache on the GPU: rows quantised as they are written, read back,
and nothing else touched."""
from __future__ import annotations

import numpy as np
import pytest

from attn_helpers import TINY, TOP, Batch, torch_type

pytestmark = pytest.mark.gpu

SHAPES = [
    # lens, kv heads, dim, page
    ([(1, 1)], 1, 64, 16),
    ([(1, 17), (3, 3), (0, 9), (16, 33)], 2, 128, 16),
    ([(5, 300), (130, 130), (1, 257)], 3, 64, 64),
    ([(7, 7), (129, 400)], 8, 128, 256),
    ([(2, 2)] * 40 + [(0, 0)] * 3 + [(1, 50)] * 33, 5, 128, 32),
]


def new_rows(b):
    import torch
    cut = [(x[kv - n:], y[kv - n:]) for (n, kv), x, y in zip(b.lens, b.k_seq, b.v_seq)]
    return (torch.cat([x for x, _ in cut]).to(b.device), torch.cat([y for _, y in cut]).to(b.device))


def quantised(x, kind):
    """Codes (as numbers) and scales of rows in fp32, step by step as defined."""
    x = x.float().cpu().numpy().astype(np.float32)
    a = np.maximum(np.abs(x).max(-1), np.float32(TINY))
    inv = np.float32(TOP[kind]) / a
    y = x * inv[..., None]
    if kind == "int8":
        code = np.rint(y)
    else:
        _, e = np.frexp(y)
        step = np.ldexp(np.float32(1), np.maximum(e - 1, -6) - 3).astype(np.float32)
        code = np.rint(y / step) * step
    return code.astype(np.float32), a / np.float32(TOP[kind])


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_write_and_read(shape, kind):
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    lens, heads, dim, page = SHAPES[shape]
    b = Batch(lens, heads, heads, dim, page, kind, seed=shape)
    before = [t.clone() for t in b.cache if t is not None]
    k, v = new_rows(b)
    pkg.ssd_kv_cache_write(k, v, *b.cache, *b.where, errors=b.errors)
    back = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    pkg.ssd_kv_cache_read(*back, *b.cache, *b.where, errors=b.errors)
    assert b.errors.item() == 0
    owned = np.zeros((b.pages, heads, page), bool)
    at = 0
    for s, (n, kv) in enumerate(lens):
        for i in range(n):
            p, r = b.row_of(s, kv - n + i)
            owned[p, :, r] = True
            for name, x, y in (("k", k, back[0]), ("v", v, back[1])):
                got = getattr(b, name + "_cache")[p, :, r]
                if kind == "bf16":
                    assert torch.equal(got, x[at]) and torch.equal(y[at], x[at])
                    continue
                code, scale = quantised(x[at], kind)
                gs = getattr(b, name + "_scale")[p, :, r].cpu().numpy()
                gc = got.float().cpu().numpy()
                assert np.array_equal(gs, scale)
                assert np.array_equal(gc, code)
                want = torch.from_numpy(gc * gs[:, None]).bfloat16()
                assert torch.equal(y[at].cpu(), want)
                # against the value itself in 64 bits: half a step of the code
                x64 = x[at].double().cpu().numpy()
                step = 1.0 if kind == "int8" else np.maximum(2.0 ** -9, np.abs(code) * 2.0 ** -3)
                err = np.abs(gc.astype(np.float64) * gs[:, None].astype(np.float64) - x64)
                assert np.all(err <= 0.5 * step * gs[:, None] * (1 + 2.0 ** -6))
            at += 1
    # every other row of the cache is as it was
    mask = torch.from_numpy(~owned).to(b.device)
    after = [t for t in b.cache if t is not None]
    for x, y in zip(before, after):
        ints = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[x.element_size()]
        assert torch.equal(x.view(ints)[mask], y.view(ints)[mask])


@pytest.mark.parametrize("kind", ["fp8", "int8"])
def test_extreme_rows(kind):
    """Rows of zeros, of the smallest and largest numbers, and of infinities and
    NaN: the last read back as NaN, the others within half a step."""
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    b = Batch([(12, 12)], 2, 2, 64, 16, kind, seed=5)
    k, v = new_rows(b)
    k[0] = 0.0
    k[1] = torch.tensor(2.0 ** -133)          # a bf16 subnormal
    k[2, :, 3] = 3.3895e38                    # the largest bf16
    k[3, 0, 9] = float("inf")
    k[4, 1, 63] = float("nan")
    k[5, 0, 0] = -float("inf")
    k[6] *= 2.0 ** -80
    v[7] = -v[7].abs().amax()
    pkg.ssd_kv_cache_write(k, v, *b.cache, *b.where, errors=b.errors)
    rk, rv = torch.empty_like(k), torch.empty_like(v)
    pkg.ssd_kv_cache_read(rk, rv, *b.cache, *b.where, errors=b.errors)
    bad = torch.zeros(12, 2, dtype=torch.bool, device=k.device)
    bad[3, 0] = bad[4, 1] = bad[5, 0] = True
    assert torch.equal(torch.isnan(rk).all(-1), bad) and torch.equal(torch.isnan(rk).any(-1), bad)
    assert torch.isfinite(rv).all()
    assert (rk[0] == 0).all() and (rk[1] == 0).all()
    # below 2^-60 the step is that of a row whose largest is 2^-60
    step = (1.0 if kind == "int8" else 2.0 ** -9) * TINY / TOP[kind]
    assert ((rk[6].double() - k[6].double()).abs() <= 0.5 * step * (1 + 2.0 ** -6)).all()
    assert torch.isfinite(rk[2]).all() and rk[2, 0, 3] > 3.38e38
    assert torch.equal(rv[7], v[7])           # a row of one magnitude is its scale times M
    assert b.errors.item() == 0


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_strided_rows(kind):
    """k and v as column slices of one fused projection, and read back into slices."""
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    b = Batch([(9, 40), (33, 33)], 4, 4, 64, 32, kind, seed=6)
    k, v = new_rows(b)
    plain = Batch([(9, 40), (33, 33)], 4, 4, 64, 32, kind, seed=6)
    pkg.ssd_kv_cache_write(k, v, *plain.cache, *plain.where)
    wide = torch.randn(b.total, 3 * 4 * 64 + 8, device="cuda").bfloat16()
    ks, vs = wide[:, 256:512].view(b.total, 4, 64), wide[:, 520:776].view(b.total, 4, 64)
    ks.copy_(k)
    vs.copy_(v)
    kept = wide.clone()
    pkg.ssd_kv_cache_write(ks, vs, *b.cache, *b.where)
    for x, y in zip(plain.cache, b.cache):
        assert x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert torch.equal(kept, wide)
    ks.zero_()
    vs.zero_()
    pkg.ssd_kv_cache_read(ks, vs, *b.cache, *b.where)
    rk, rv = torch.empty_like(k), torch.empty_like(v)
    pkg.ssd_kv_cache_read(rk, rv, *plain.cache, *plain.where)
    assert torch.equal(ks, rk) and torch.equal(vs, rv)
    kept[:, 256:512], kept[:, 520:776] = ks.flatten(1), vs.flatten(1)
    assert torch.equal(kept, wide)


def test_padding_rows():
    """Rows at a negative position are not written and read back as zeros."""
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    b = Batch([(4, 4), (1, 1)], 2, 2, 64, 16, "int8", seed=7)
    k, v = new_rows(b)
    pkg.ssd_kv_cache_write(k, v, *b.cache, *b.where)
    kept = [t.clone() for t in b.cache]
    b.kv_lens.copy_(torch.tensor([1, 0]))
    rows = torch.ones_like(k), torch.ones_like(v)
    pkg.ssd_kv_cache_read(*rows, *b.cache, *b.where, errors=b.errors)
    for r in rows:
        assert (r[[0, 1, 2, 4]] == 0).all() and (r[3] != 0).any()
    pkg.ssd_kv_cache_write(k + 1, v + 1, *b.cache, *b.where, errors=b.errors)
    p, r = b.row_of(0, 0)
    for x, y in zip(kept, b.cache):
        same = (x.view(torch.uint8) == y.view(torch.uint8)).view(b.pages, 2, 16, -1).all(-1)
        same[p, :, r] = True
        assert same.all()
    assert b.errors.item() == 0


def test_device_side_errors():
    """Bad pages, lengths and offsets are flagged, skipped and read as zeros."""
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    from mamba_ssd_chunked_varlen_gb300 import attention, binding

    def make():
        b = Batch([(20, 20), (3, 3)], 2, 2, 64, 16, "bf16", seed=8)
        return b, *new_rows(b)

    for bad in (-1, 1 << 20):
        b, k, v = make()
        b.block_table[0, 1] = bad
        before = b.k_cache.clone()
        pkg.ssd_kv_cache_write(k, v, *b.cache, *b.where, errors=b.errors)
        assert b.errors.item() == attention.DEVERR_BAD_PAGE
        rk, rv = torch.ones_like(k), torch.ones_like(v)
        pkg.ssd_kv_cache_read(rk, rv, *b.cache, *b.where)
        assert torch.equal(rk[:16], k[:16]) and (rk[16:20] == 0).all() and torch.equal(rk[20:], k[20:])
        changed = (before.view(torch.int16) != b.k_cache.view(torch.int16)).any(-1).sum()
        assert changed == 2 * (16 + 3)
    for n in (-1, 1000):
        b, k, v = make()
        b.kv_lens[1] = n
        pkg.ssd_kv_cache_write(k, v, *b.cache, *b.where, errors=b.errors)
        assert b.errors.item() == attention.DEVERR_BAD_KV_LEN
        rk, rv = torch.ones_like(k), torch.ones_like(v)
        pkg.ssd_kv_cache_read(rk, rv, *b.cache, *b.where)
        assert torch.equal(rk[:20], k[:20]) and (rk[20:] == 0).all()
    for q in ([0, 20, 22], [1, 20, 23], [0, 25, 23]):
        b, k, v = make()
        b.query_start_loc.copy_(torch.tensor(q))
        rk, rv = torch.ones_like(k), torch.ones_like(v)
        pkg.ssd_kv_cache_read(rk, rv, *b.cache, *b.where, errors=b.errors)
        assert b.errors.item() & binding.DEVERR_BAD_QUERY_START_LOC


def test_far_pages():
    """A row past 2^31 elements into the cache."""
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    pages = (1 << 31) // (256 * 2 * 64) + 3
    k_cache = torch.zeros((pages, 2, 256, 64), dtype=torch.int8, device="cuda")
    v_cache = torch.zeros_like(k_cache)
    k_scale = torch.zeros((pages, 2, 256), device="cuda")
    v_scale = torch.zeros_like(k_scale)
    k = torch.randn(300, 2, 64, device="cuda").bfloat16()
    where = (torch.tensor([0, 300], dtype=torch.int32, device="cuda"),
             torch.tensor([300], dtype=torch.int32, device="cuda"),
             torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda"))
    pkg.ssd_kv_cache_write(k, k, k_cache, v_cache, k_scale, v_scale, *where)
    code, scale = quantised(k, "int8")
    assert np.array_equal(k_cache[pages - 1].permute(1, 0, 2).float().cpu().numpy(), code[:256])
    assert np.array_equal(v_scale[pages - 2, :, :44].T.cpu().numpy(), scale[256:])
    assert not k_cache[:pages - 2].any()
