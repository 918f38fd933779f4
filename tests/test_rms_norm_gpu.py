"""The root-mean-square norm on the GPU against the formula in 64 bits.

Relative bound of y before its output type: s is rounded once (a gate's silu adds
2^-21 + |z| 2^-23 and two roundings); that moves the mean's root by as much again; a
thread adds at most 32 squares, its lane's and its warp's sums follow in ten steps
(42 roundings, half of which the root keeps), the root is off by 2^-22 and two
products follow.  bf16 adds half a step of 2^-8.  A code is off by half its step and
the scale by y's bound."""
from __future__ import annotations

import numpy as np
import pytest

from layer_helpers import E, U, f64, near, same_bits, sliced

pytestmark = pytest.mark.gpu

TOP = {"int8": 127.0, "fp8": 448.0}
TINY = 2.0 ** -60


def norm_ref(x, weight, residual, gate, groups, eps):
    """s, y in 64 bits and y's relative bound before it is rounded to its type."""
    s, off = x, E
    if residual is not None:
        s = x + residual
    if gate is not None:
        s = x * (gate / (1 + np.exp(-gate)))
        off = 2.0 ** -21 + np.abs(np.where(np.isfinite(gate), gate, 0)).max() * 2.0 ** -23 + 3 * E
    g = s.reshape(s.shape[0], groups, -1)
    y = (g / np.sqrt((g * g).mean(-1, keepdims=True) + eps)).reshape(s.shape)
    return s, y * weight, 2 * off + 21 * E + 2.0 ** -22 + 3 * E


def run(rows, dim, kind="bf16", groups=1, residual=False, gate=False, weight=True, eps=1e-5, seed=0,
        strided=False, change=None, scale_by=1.0, stream=None):
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    gen = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen)

    x = (normal(rows, dim) * scale_by).bfloat16().cuda()
    r = (normal(rows, dim) * scale_by).bfloat16().cuda() if residual else None
    z = normal(rows, dim).bfloat16().cuda() if gate else None
    w = (1 + 0.3 * normal(dim)).cuda() if weight else None
    if change:
        change(x, r)
    before = [None if t is None else t.clone() for t in (x, r, z)]
    kind_t = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "int8": torch.int8}[kind]
    y = torch.zeros(rows, dim, device="cuda").to(kind_t)
    scale = torch.zeros(rows, groups, device="cuda") if kind != "bf16" else None
    args, wides = [x, r, z], []
    if strided:
        args = []
        for t in (x, r, z):
            wide, view = (None, None) if t is None else sliced(t)
            wides.append((wide, None if wide is None else wide.clone()))
            args.append(view)
    pkg.ssd_rms_norm_fwd(y, args[0], w, residual=args[1], gate=args[2], scale=scale, ngroups=groups,
                         eps=eps, stream=stream)
    torch.cuda.synchronize()
    xb, rb, zb = (None if t is None else f64(t) for t in before)
    s, want, rel = norm_ref(xb, f64(w) if weight else 1.0, rb, zb, groups, eps)
    if residual:
        assert same_bits(args[1], (before[0].float() + before[1].float()).bfloat16())
    if strided:
        for (wide, kept), t, name in zip(wides, args, ("x", "residual", "gate")):
            if wide is not None:
                kept[:, 16:-16] = t
                assert same_bits(wide, kept), name
    if kind == "bf16":
        near(f64(y), want, np.abs(want) * (U + rel * (1 + U)) + 2.0 ** -133, "y")
        return y
    code, sc = f64(y).reshape(rows, groups, -1), f64(scale)
    want = want.reshape(rows, groups, -1)
    a = np.abs(want).max(-1)
    bad = ~np.isfinite(a)
    assert np.array_equal(np.isnan(sc), bad) and (code[bad] == 0).all()
    a = np.maximum(np.where(bad, 0, a), TINY)
    near(sc[~bad], a[~bad] / TOP[kind], a[~bad] / TOP[kind] * (rel + 2 * E), "scale")
    step = 1.0 if kind == "int8" else np.maximum(2.0 ** -9, np.abs(code) * 2.0 ** -3)
    got, want = code * np.where(bad, 0, sc)[..., None], np.where(bad[..., None], 0, want)
    near(got, want, 0.5 * step * np.where(bad, 0, sc)[..., None] * (1 + 2.0 ** -6) + np.abs(want) * 2 * rel, "y")
    assert np.abs(code).max() <= TOP[kind]
    return y, scale


COLS = [8, 16, 56, 64, 72, 120, 128, 136, 248, 256, 264, 512, 520, 1000, 1024, 1032, 2048, 4096, 5120, 16384, 16392, 32768]


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("kind", ["bf16", "fp8", "int8"])
def test_columns(cols, kind):
    run(5, cols, kind, residual=True, seed=cols)
    run(1, cols, kind, seed=cols)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("groups,cols", [(1, 1024), (8, 1024), (3, 40), (2, 2048), (5, 264)])
def test_gate_and_groups(kind, groups, cols):
    run(7, groups * cols, kind, groups, gate=True, seed=groups)
    run(6, groups * cols, kind, groups, weight=False, seed=groups)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int8"])
def test_strided(kind):
    run(9, 520, kind, residual=True, strided=True)
    run(9, 2 * 1040, kind, 2, gate=True, strided=True)


@pytest.mark.parametrize("rows", [1, 3, 151, 4093])
def test_rows(rows):
    run(rows, 64, residual=True)
    run(rows, 1536, "int8", residual=True)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("cols", [64, 128, 256, 4096])
def test_ranges(kind, cols):
    """Squares beyond fp32's range, values far below eps, zeros, infinities and NaN:
    a row's own alone."""
    run(4, cols, kind, scale_by=2.0 ** 100, residual=True)
    run(7, cols, kind, scale_by=2.0 ** 70, change=lambda x, r: x[::2].mul_(2.0 ** -70))
    run(4, cols, kind, scale_by=2.0 ** -60, eps=2.0 ** -80)
    run(4, cols, kind, scale_by=2.0 ** -90)

    def change(x, r):
        x[0] = 0
        r[0] = 0
        x[1] = 0
        x[2, 7] = float("inf")
        x[3, cols - 1] = float("nan")
        x[4, 3] = 3.0e38
        x[5, 9] = -float("inf")
        r[6, 11] = float("inf")
        x[6, 11] = -float("inf")
    run(9, cols, kind, residual=True, change=change)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("rows,groups,cols", [(701, 3, 1040), (1500, 1, 1096), (333, 1, 16384), (160, 5, 8200), (3, 200, 1032)])
def test_rows_in_turn(kind, rows, groups, cols):
    """More rows than CTAs at once, more groups than these, and rows of infinities, NaN and
    squares out of range between others."""
    def change(x, r):
        for at, value in ((5, float("inf")), (rows // 2, 3.0e38), (rows // 2 + 1, 2.0e38), (rows - 2, float("nan"))):
            if 0 <= at < rows:
                x[at, at % cols] = value
    run(rows, groups * cols, kind, groups, gate=True, seed=rows)
    run(rows, groups * cols, kind, groups, residual=groups == 1, seed=rows, change=change if rows > 100 else None)


@pytest.mark.parametrize("gate", [False, True])
def test_rows_in_turn_in_place(gate):
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    x, z = torch.randn(2, 1100, 2 * 1160, device="cuda").bfloat16().unbind()
    w = torch.randn(2 * 1160, device="cuda")
    y = torch.empty_like(x)
    pkg.ssd_rms_norm_fwd(y, x, w, gate=z if gate else None, ngroups=2)
    for take in range(1 + gate):
        args = [x.clone(), z.clone()]
        pkg.ssd_rms_norm_fwd(args[take], args[0], w, gate=args[1] if gate else None, ngroups=2)
        assert same_bits(args[take], y)


def test_in_place():
    """y may be x or the gate."""
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    x, z = torch.randn(2, 33, 4 * 520, device="cuda").bfloat16().unbind()
    w = torch.randn(4 * 520, device="cuda")
    y = torch.empty_like(x)
    pkg.ssd_rms_norm_fwd(y, x, w, gate=z, ngroups=4)
    for take in (0, 1):
        args = [x.clone(), z.clone()]
        pkg.ssd_rms_norm_fwd(args[take], args[0], w, gate=args[1], ngroups=4)
        assert same_bits(args[take], y)


def test_stream_and_graph():
    import torch
    import mamba_ssd_chunked_varlen_gb300 as pkg
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    run(33, 1032, "int8", residual=True, stream=stream)
    x, w = torch.randn(5, 2048, device="cuda").bfloat16(), torch.randn(2048, device="cuda")
    r, y = torch.zeros_like(x), torch.empty_like(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.ssd_rms_norm_fwd(y, x, w, residual=r)
    r.zero_()
    for _ in range(2):
        kept, want = r.clone(), torch.empty_like(y)
        graph.replay()
        pkg.ssd_rms_norm_fwd(want, x, w, residual=kept)
        torch.cuda.synchronize()
        assert same_bits(y, want) and same_bits(r, kept)
