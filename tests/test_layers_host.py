"""Host-side checks of include/ssd_layers.h (no GPU): header and binding agree, and
bad arguments are refused before any launch."""
from __future__ import annotations

import ctypes
import os
import re

import pytest

from mamba_ssd_chunked_varlen_gb300 import binding, layers
from mamba_ssd_chunked_varlen_gb300 import build as cuda_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 12      # an aligned address that no refused call touches


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    layers._functions()
    return binding.library()


def _vp(v):
    return None if v is None else ctypes.c_void_p(v)


def test_header_and_binding_agree(lib):
    text = open(os.path.join(ROOT, "include", "ssd_layers.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    declared = sorted(set(re.findall(r"\b(ssd_\w+)\s*\(", text)))
    assert declared == sorted(layers.EXPORTED_SYMBOLS)
    for name in declared:
        assert hasattr(lib, name)


def _conv(lib, **over):
    a = dict(y=A, x=A, weight=A, bias=None, pool=A, qsl=A, has=None, slots=A, total=10, batch=2,
             channels=64, width=4, max_slots=4, ys=0, xs=0) | over
    return lib.ssd_causal_conv_varlen_fwd(
        _vp(a["y"]), _vp(a["x"]), _vp(a["weight"]), _vp(a["bias"]), _vp(a["pool"]), _vp(a["qsl"]),
        _vp(a["has"]), _vp(a["slots"]), a["total"], a["batch"], a["channels"], a["width"],
        a["max_slots"], a["ys"], a["xs"], 1, None, None)


@pytest.mark.parametrize("over,status", [
    (dict(total=-1), 1), (dict(batch=-1), 1), (dict(max_slots=-1), 1), (dict(channels=0), 1),
    (dict(width=0), 1), (dict(y=None), 1), (dict(x=None), 1), (dict(weight=None), 1),
    (dict(pool=None), 1), (dict(qsl=None), 1), (dict(slots=None), 1), (dict(x=A + 8), 1),
    (dict(y=A + 2), 1), (dict(weight=A + 4), 1), (dict(bias=A + 4), 1), (dict(pool=A + 8), 1),
    (dict(ys=56), 1), (dict(xs=68), 1),
    (dict(width=1), 2), (dict(width=5), 2), (dict(channels=60), 2), (dict(channels=(1 << 20) + 8), 2),
    (dict(total=1 << 31), 2), (dict(batch=(1 << 31) - 1), 2),
    (dict(batch=0), 0), (dict(batch=0, total=0, x=None, y=None, qsl=None, slots=None), 0),
])
def test_conv_refuses(lib, over, status):
    assert _conv(lib, **over) == status


def test_binding_refuses_cpu_tensors(lib):
    import torch
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        layers.ssd_causal_conv_varlen_fwd(x, x, torch.zeros(64, 4), None, x.view(1, 2, 64), i, None, i[:1])


def _norm(lib, **over):
    a = dict(y=A, scale=None, x=A, residual=None, gate=None, weight=A, rows=4, dim=64, groups=1, kind=0,
             eps=1e-5, ys=0, xs=0, rs=0, gs=0) | over
    return lib.ssd_rms_norm_fwd(
        _vp(a["y"]), _vp(a["scale"]), _vp(a["x"]), _vp(a["residual"]), _vp(a["gate"]), _vp(a["weight"]),
        a["rows"], a["dim"], a["groups"], a["kind"], a["eps"], a["ys"], a["xs"], a["rs"], a["gs"], None)


@pytest.mark.parametrize("over,status", [
    (dict(rows=-1), 1), (dict(dim=0), 1), (dict(groups=0), 1), (dict(groups=3), 1), (dict(kind=3), 1),
    (dict(kind=-1), 1), (dict(eps=0.0), 1), (dict(eps=-1.0), 1), (dict(eps=2.0), 1),
    (dict(eps=float("nan")), 1), (dict(y=None), 1), (dict(x=None), 1), (dict(kind=1), 1),
    (dict(kind=2), 1), (dict(scale=A), 1), (dict(residual=A, gate=A), 1), (dict(x=A + 8), 1),
    (dict(y=A + 8), 1), (dict(residual=A + 2), 1), (dict(gate=A + 4), 1), (dict(weight=A + 4), 1),
    (dict(ys=56), 1), (dict(xs=68), 1), (dict(rs=8), 1), (dict(gs=65), 1),
    (dict(groups=16), 2), (dict(dim=60), 2), (dict(dim=32768 + 8), 2), (dict(rows=1 << 31), 2),
    (dict(rows=1 << 29, dim=64 * 64, groups=64), 2), (dict(rows=0, y=None, x=None), 0),
])
def test_norm_refuses(lib, over, status):
    assert _norm(lib, **over) == status


ROPE = dict(qo=A, q=A, ko=A, k=A, v=A, turns=A, qsl=A, kv_lens=A, total=10, batch=2, heads=4, kv_heads=2, dim=64,
            part=64, inter=0, m=1.0, qos=0, qs=0, kos=0, ks=0, vs=0, k_cache=A, v_cache=A, k_scale=None,
            v_scale=None, table=A, pages=8, page=16, width=4, stride=4, kind=0)


def _rope(lib, **over):
    a = ROPE | over
    return lib.ssd_rope_varlen_fwd(
        _vp(a["qo"]), _vp(a["q"]), _vp(a["ko"]), _vp(a["k"]), _vp(a["turns"]), _vp(a["qsl"]), _vp(a["kv_lens"]),
        a["total"], a["batch"], a["heads"], a["kv_heads"], a["dim"], a["part"], a["inter"], a["m"], a["qos"],
        a["qs"], a["kos"], a["ks"], None, None)


def _rope_write(lib, **over):
    a = ROPE | over
    return lib.ssd_rope_kv_cache_write(
        _vp(a["qo"]), _vp(a["q"]), _vp(a["k"]), _vp(a["v"]), _vp(a["turns"]), _vp(a["k_cache"]), _vp(a["v_cache"]),
        _vp(a["k_scale"]), _vp(a["v_scale"]), _vp(a["qsl"]), _vp(a["kv_lens"]), _vp(a["table"]), a["total"],
        a["batch"], a["heads"], a["kv_heads"], a["dim"], a["part"], a["inter"], a["m"], a["pages"], a["page"],
        a["width"], a["stride"], a["kind"], a["qos"], a["qs"], a["ks"], a["vs"], None, None)


@pytest.mark.parametrize("over,status", [
    (dict(total=-1), 1), (dict(batch=-1), 1), (dict(dim=0), 1), (dict(heads=-1), 1), (dict(part=0), 1),
    (dict(part=80), 1), (dict(m=float("nan")), 1), (dict(m=float("inf")), 1), (dict(turns=None), 1),
    (dict(turns=A + 4), 1), (dict(q=None), 1), (dict(qo=None), 1), (dict(k=None), 1), (dict(qsl=None), 1),
    (dict(kv_lens=None), 1), (dict(q=A + 8), 1), (dict(qo=A + 2), 1), (dict(k=A + 8), 1), (dict(qs=248), 1),
    (dict(qos=260), 1), (dict(ks=8), 1), (dict(part=8), 2), (dict(part=24), 2), (dict(dim=96), 2),
    (dict(total=1 << 31), 2), (dict(heads=1 << 16), 2), (dict(kv_heads=1 << 16), 2),
    (dict(total=0, q=None, k=None, v=None), 0),
])
def test_rope_refuses(lib, over, status):
    assert _rope(lib, **over) == status
    assert _rope_write(lib, **over) == status


def test_rope_refuses_more(lib):
    assert _rope(lib, ko=None) == 1
    assert _rope(lib, ko=A + 4) == 1
    assert _rope(lib, kos=120) == 1
    assert _rope(lib, heads=0, kv_heads=0) == 1
    assert _rope(lib, batch=0) == 0                  # a padded batch without sequences
    assert _rope_write(lib, batch=0) == 0
    for over, status in ((dict(v=None), 1), (dict(v=A + 8), 1), (dict(vs=120), 1), (dict(heads=0), 1),
                         (dict(kv_heads=0), 1), (dict(k_cache=None), 1), (dict(table=None), 1), (dict(kind=1), 1),
                         (dict(kind=3), 1), (dict(page=48), 2), (dict(stride=3), 1), (dict(pages=0), 1)):
        assert _rope_write(lib, **over) == status, over


def test_rope_table_refuses(lib):
    for f in (-1.0, 6.3, float("nan"), float("inf")):
        with pytest.raises(binding.SSDError):
            layers.alloc_rope_table([1.0, f], "cpu")
    with pytest.raises(ValueError):
        layers.alloc_rope_table([], "cpu")
    assert lib.ssd_rope_table(None, None, 0) == 0
    assert lib.ssd_rope_table(None, None, 1) == 1
    assert lib.ssd_rope_table(None, None, -1) == 1


def test_rope_frequencies():
    import math
    f = layers.rope_frequencies
    plain, m = f(64, 10000.0)
    assert m == 1.0 and len(plain) == 32 and plain[0] == 1.0
    assert math.isclose(plain[31], 10000.0 ** (-62 / 64), rel_tol=1e-12)
    assert f(64, scaling="linear", factor=4.0) == ([x / 4.0 for x in plain], 1.0)
    based, m = f(64, scaling="base", factor=4.0)
    assert m == 1.0 and based[0] == 1.0 and math.isclose(based[31], plain[31] / 4.0, rel_tol=1e-12)
    for scaling, low, high in (("ramp", 1.0, 32.0), ("wavelength", 1.0, 4.0)):
        got, m = f(64, scaling=scaling, factor=8.0, original_len=2048, low_turns=low, high_turns=high)
        assert m == (0.1 * math.log(8.0) + 1.0 if scaling == "ramp" else 1.0)
        for x, y in zip(plain, got):
            turns = x * 2048 / (2 * math.pi)
            assert x / 8.0 * (1 - 1e-12) <= y <= x
            if turns >= 2 * high:
                assert y == x
            if turns <= low / 2:
                assert math.isclose(y, x / 8.0, rel_tol=1e-12)
        assert f(64, scaling=scaling, factor=1.0)[0] == pytest.approx(plain, rel=1e-12)
    for bad in (dict(rotary_dim=63), dict(rotary_dim=2), dict(rotary_dim=64, base=1.0),
                dict(rotary_dim=64, factor=0.5), dict(rotary_dim=64, scaling="other"),
                dict(rotary_dim=64, scaling="ramp", low_turns=4.0, high_turns=2.0)):
        with pytest.raises(ValueError):
            f(**bad)


@pytest.mark.parametrize("rotary_dim,base,original_len,low,high", [
    (128, 1e4, 65536, 1.0, 32.0), (128, 1e4, 131072, 1.0, 32.0), (64, 1e4, 131072, 1.0, 32.0),
    (64, 1e4, 1 << 24, 1.0, 32.0),               # the ramp's end behind rotary_dim - 1
    (64, 1e4, 1 << 28, 1.0, 32.0),               # all pairs make more than high_turns
    (128, 1e6, 32768, 1.0, 32.0), (64, 1e4, 8192, 1.0, 32.0), (32, 1e4, 8192, 0.5, 4.0),
    (64, 1e4, 200, 1.0, 32.0), (64, 1e4, 6, 1.0, 32.0), (64, 1e4, 3, 1.0, 32.0),
])
def test_rope_ramp(rotary_dim, base, original_len, low, high):
    """The share of the plain frequency by the definition, with the pairs' turns counted."""
    import math
    factor, half = 8.0, rotary_dim // 2
    plain, _ = layers.rope_frequencies(rotary_dim, base)
    got, _ = layers.rope_frequencies(rotary_dim, base, scaling="ramp", factor=factor, original_len=original_len,
                                     low_turns=low, high_turns=high)

    # pair i makes original_len base^(-i / half) / (2 pi) turns: where that is high, and low
    def index(turns):
        return half * math.log(original_len / (2 * math.pi * turns), base)
    start, end = max(math.floor(index(high)), 0), min(math.ceil(index(low)), rotary_dim - 1)
    for i, (x, y) in enumerate(zip(plain, got)):
        turns = original_len * x / (2 * math.pi)
        keep = (y / x * factor - 1.0) / (factor - 1.0)
        if turns <= low:
            assert keep == pytest.approx(0.0, abs=1e-12)
        elif turns >= high:
            assert keep == pytest.approx(1.0, abs=1e-12)
        else:
            assert keep == pytest.approx(min(max((end - i) / (end - start), 0.0), 1.0), abs=1e-9)


def test_rope_binding_refuses(lib):
    import torch
    q = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    table = layers.alloc_rope_table([1.0] * 32, "cpu")
    assert table.dtype == torch.int64 and table.shape == (32,)
    with pytest.raises(ValueError):
        layers.ssd_rope_varlen_fwd(None, None, None, None, table, i, i[:1])
    with pytest.raises(ValueError):
        layers.ssd_rope_varlen_fwd(q, q, None, q, table, i, i[:1])
    with pytest.raises(ValueError):
        layers.ssd_rope_varlen_fwd(q, q, None, None, table, i, i[:1])     # CPU tensors


def _scan(lib, **over):
    a = dict(y=A, x=A, dt=A, A=A, B=A, C=A, D=None, z=None, bias=None, pool=A, qsl=A, has=None, slots=A,
             total=10, batch=2, channels=64, dstate=16, max_slots=4, pool_type=0, strides={}, ws=A,
             wsb=1 << 40) | over
    return lib.ssd_selective_scan_varlen_fwd(
        _vp(a["y"]), _vp(a["x"]), _vp(a["dt"]), _vp(a["A"]), _vp(a["B"]), _vp(a["C"]), _vp(a["D"]), _vp(a["z"]),
        _vp(a["bias"]), _vp(a["pool"]), _vp(a["qsl"]), _vp(a["has"]), _vp(a["slots"]), a["total"], a["batch"],
        a["channels"], a["dstate"], a["max_slots"], a["pool_type"], 1,
        None if a["strides"] is None else ctypes.byref(layers.SelectiveStrides(**a["strides"])), _vp(a["ws"]),
        a["wsb"], None, None)


@pytest.mark.parametrize("over,status", [
    (dict(total=-1), 1), (dict(batch=-1), 1), (dict(max_slots=-1), 1), (dict(channels=0), 1),
    (dict(dstate=0), 1), (dict(pool_type=2), 1), (dict(pool_type=-1), 1), (dict(y=None), 1), (dict(x=None), 1),
    (dict(dt=None), 1), (dict(A=None), 1), (dict(B=None), 1), (dict(C=None), 1), (dict(pool=None), 1),
    (dict(qsl=None), 1), (dict(slots=None), 1), (dict(x=A + 8), 1), (dict(y=A + 2), 1), (dict(dt=A + 2), 1),
    (dict(z=A + 8), 1), (dict(B=A + 8), 1), (dict(C=A + 4), 1), (dict(A=A + 4), 1), (dict(pool=A + 8), 1),
    (dict(strides=dict(x=56)), 1), (dict(strides=dict(y=68)), 1), (dict(strides=dict(dt=65)), 1),
    (dict(strides=dict(B=8)), 1), (dict(strides=dict(C=20)), 1), (dict(strides=dict(z=-64)), 1),
    (dict(channels=60), 2), (dict(channels=(1 << 20) + 8), 2), (dict(dstate=4), 2), (dict(dstate=24), 2),
    (dict(dstate=128), 2), (dict(strides=dict(dt=1 << 31)), 2), (dict(total=1 << 31), 2), (dict(batch=(1 << 31) - 1), 2),
    (dict(ws=None), 3), (dict(ws=A + 16), 3), (dict(wsb=16), 3),
    (dict(batch=0), 0), (dict(batch=0, strides=None, ws=None), 0),
])
def test_scan_refuses(lib, over, status):
    assert _scan(lib, **over) == status


def test_scan_workspace_size(lib):
    size = layers.ssd_selective_scan_varlen_workspace_size
    assert size(0, 0, 8, 8) > 0 and size(1, 1, 64, 16) > 0
    for bad in ((-1, 1, 64, 16), (1, -1, 64, 16), (1, 1, 60, 16), (1, 1, 64, 12), (1, 1, 0, 16), (1 << 31, 1, 64, 16)):
        assert size(*bad) == 0
    # enough for every call that is not larger in any size
    sizes = [(t, b, c, n) for t in (1, 1000, 100000) for b in (1, 64) for c in (8, 1024, 16384) for n in (8, 64)]
    for big in sizes:
        for small in sizes:
            if all(x <= y for x, y in zip(small, big)):
                assert size(*small) <= size(*big), (small, big)
