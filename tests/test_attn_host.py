"""Host-side checks of include/ssd_attn.h (no GPU): header and binding agree,
the workspace is sized, and bad arguments are refused before any launch."""
from __future__ import annotations

import ctypes
import os
import re

import pytest

from mamba_ssd_chunked_varlen_gb300 import attention, binding
from mamba_ssd_chunked_varlen_gb300 import build as cuda_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 12      # an aligned address that no refused call touches


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    attention._functions()
    return binding.library()


def test_header_and_binding_agree(lib):
    text = open(os.path.join(ROOT, "include", "ssd_attn.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    declared = sorted(set(re.findall(r"\b(ssd_\w+)\s*\(", text)))
    assert declared == sorted(attention.EXPORTED_SYMBOLS)
    for name in declared:
        assert hasattr(lib, name)


def test_workspace_size(lib):
    ws = attention.ssd_attn_varlen_workspace_size
    assert ws(1, 1, 8, 2, 128) > 0
    assert ws(0, 0, 8, 2, 128) > 0
    assert ws(100, 4, 8, 3, 128) == 0        # nheads % nheads_kv
    assert ws(100, 4, 8, 2, 80) == 0         # head_dim
    assert ws(100, 4, 256, 1, 64) == 0       # more than 128 query heads a kv head
    assert ws(-1, 4, 8, 2, 64) == 0
    assert ws(1 << 31, 4, 8, 2, 64) == 0
    # enough for every smaller call of the same heads
    assert ws(4096, 64, 8, 2, 64) >= ws(64, 64, 8, 2, 64) >= ws(1, 1, 8, 2, 64)


CACHE = dict(k_cache=A, v_cache=A, k_scale=None, v_scale=None, qsl=A, kv_lens=A, table=A,
             total=10, batch=2, kv_heads=2, dim=64, pages=8, page=16, width=4, stride=4, kind=0)


def _vp(v):
    return None if v is None else ctypes.c_void_p(v)


def _copy(fn, **over):
    a = dict(CACHE, k=A, v=A, ks=0, vs=0) | over
    return fn(_vp(a["k"]), _vp(a["v"]), _vp(a["k_cache"]), _vp(a["v_cache"]), _vp(a["k_scale"]),
              _vp(a["v_scale"]), _vp(a["qsl"]), _vp(a["kv_lens"]), _vp(a["table"]), a["total"],
              a["batch"], a["kv_heads"], a["dim"], a["pages"], a["page"], a["width"], a["stride"],
              a["kind"], a["ks"], a["vs"], None, None)


def _attn(lib, **over):
    a = dict(CACHE, o=A, lse=None, q=A, heads=4, os=0, qs=0, scale=0.1, window=0, ws=A,
             wsb=1 << 40) | over
    return lib.ssd_attn_varlen_fwd(
        _vp(a["o"]), _vp(a["lse"]), _vp(a["q"]), _vp(a["k_cache"]), _vp(a["v_cache"]),
        _vp(a["k_scale"]), _vp(a["v_scale"]), _vp(a["qsl"]), _vp(a["kv_lens"]), _vp(a["table"]),
        a["total"], a["batch"], a["heads"], a["kv_heads"], a["dim"], a["pages"], a["page"],
        a["width"], a["stride"], a["kind"], a["os"], a["qs"], a["scale"], a["window"],
        _vp(a["ws"]), a["wsb"], None, None)


REFUSED = [
    (dict(total=-1), 1), (dict(batch=-1), 1), (dict(kv_heads=0), 1), (dict(dim=0), 1),
    (dict(page=0), 1), (dict(pages=-1), 1), (dict(pages=0), 1), (dict(kind=3), 1), (dict(kind=-1), 1),
    (dict(qsl=None), 1), (dict(kv_lens=None), 1), (dict(table=None), 1), (dict(k_cache=None), 1),
    (dict(v_cache=None), 1), (dict(kind=1), 1), (dict(kind=2, k_scale=A), 1),
    (dict(k_cache=A + 8), 1), (dict(v_cache=A + 2), 1), (dict(kind=1, k_scale=A, v_scale=A + 4), 1),
    (dict(stride=3), 1), (dict(batch=0), 1),
    (dict(dim=80), 2), (dict(dim=256), 2), (dict(page=8), 2), (dict(page=48), 2),
    (dict(page=512), 2), (dict(width=1 << 28), 1), (dict(width=1 << 28, stride=1 << 28), 2),
    (dict(total=1 << 31), 2),
]


@pytest.mark.parametrize("over,status", REFUSED)
def test_all_calls_refuse(lib, over, status):
    for fn in (lib.ssd_kv_cache_write, lib.ssd_kv_cache_read):
        assert _copy(fn, **over) == status
    assert _attn(lib, **over) == status


def test_copies_refuse(lib):
    for fn in (lib.ssd_kv_cache_write, lib.ssd_kv_cache_read):
        assert _copy(fn, k=None) == 1
        assert _copy(fn, v=A + 8) == 1
        assert _copy(fn, ks=127) == 1            # less than a row
        assert _copy(fn, vs=132) == 1            # not a multiple of 8
        assert _copy(fn, total=0, k=None, v=None) == 0   # nothing to do


def test_attention_refuses(lib):
    assert _attn(lib, o=None) == 1
    assert _attn(lib, q=None) == 1
    assert _attn(lib, q=A + 8) == 1
    assert _attn(lib, o=A + 2) == 1
    assert _attn(lib, heads=5) == 1
    assert _attn(lib, heads=0) == 1
    assert _attn(lib, heads=258) == 2            # 129 query heads a kv head
    assert _attn(lib, window=-1) == 1
    assert _attn(lib, scale=float("nan")) == 1
    assert _attn(lib, scale=float("inf")) == 1
    assert _attn(lib, qs=264 + 4) == 1
    assert _attn(lib, os=64) == 1
    assert _attn(lib, ws=None) == 3
    assert _attn(lib, ws=A + 16) == 3
    assert _attn(lib, wsb=16) == 3
    assert _attn(lib, total=0, q=None, o=None, ws=None, wsb=0) == 0


def test_binding_refuses_cpu_tensors(lib):
    import torch
    t = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        attention.ssd_kv_cache_write(x, x, t, t, None, None, i, i[:1], i.view(1, 2))
    with pytest.raises(ValueError):
        attention.ssd_attn_varlen_fwd(x, None, x, t, t, None, None, i, i[:1], i.view(1, 2),
                                      softmax_scale=1.0, workspace=torch.zeros(1 << 20, dtype=torch.uint8))
