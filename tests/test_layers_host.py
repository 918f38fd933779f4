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
