"""Host-side checks of the paged cache's and the attention's edges (no GPU): views
that the C ABI cannot express are refused by the binding."""
from __future__ import annotations

import pytest
import torch

from mamba_ssd_chunked_varlen_gb300 import attention


class OnDevice(torch.Tensor):
    """A CPU tensor that says it is on device 0: for checks that come before any launch."""

    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0


def on_device(t):
    return t.as_subclass(OnDevice)


@pytest.fixture
def no_launch(monkeypatch):
    """The binding with entry points that must not be reached."""
    f = attention._Functions()

    def launched(*args):
        raise AssertionError("a refused call was launched")

    f.write = f.read = f.attn = launched
    f.raw_stream = lambda device: 0
    monkeypatch.setattr(attention, "_fn", f)
    return f


def batch_of(n=2, rows=5, heads=2, dim=64, page=16, width=3):
    """Arguments of a call of `n` sequences that passes every check."""
    i32 = dict(dtype=torch.int32)
    shape = (4, heads, page, dim)
    return dict(x=on_device(torch.zeros(rows, heads, dim, dtype=torch.bfloat16)),
                cache=(on_device(torch.zeros(shape, dtype=torch.bfloat16)),
                       on_device(torch.zeros(shape, dtype=torch.bfloat16)), None, None),
                qsl=on_device(torch.zeros(n + 1, **i32)), lens=on_device(torch.zeros(n, **i32)),
                table=on_device(torch.zeros(n, width, **i32)),
                ws=on_device(torch.zeros(1024, dtype=torch.uint8)))


def calls(a, k=None, v=None, table=None, which=("write", "read", "attn")):
    """The three calls with `k` and `v` (attention: q and o) and `table` in place of the usual ones."""
    k, v = a["x"] if k is None else k, a["x"] if v is None else v
    where = (a["qsl"], a["lens"], a["table"] if table is None else table)
    made = dict(
        write=lambda: attention.ssd_kv_cache_write(k, v, *a["cache"], *where),
        read=lambda: attention.ssd_kv_cache_read(k, v, *a["cache"], *where),
        attn=lambda: attention.ssd_attn_varlen_fwd(v, None, k, *a["cache"], *where, softmax_scale=1.0,
                                                   workspace=a["ws"]))
    return [made[w] for w in which]


def test_the_usual_call_passes_the_checks(no_launch):
    for call in calls(batch_of()):
        with pytest.raises(AssertionError, match="launched"):
            call()


def overlapping(rows=5, heads=2, dim=64):
    one = torch.zeros(1, heads, dim, dtype=torch.bfloat16).expand(rows, heads, dim)
    half = torch.zeros(rows * heads * dim, dtype=torch.bfloat16).as_strided(
        (rows, heads, dim), (heads * dim // 2, dim, 1))
    return [on_device(one), on_device(half)]


@pytest.mark.parametrize("which", [0, 1])
def test_overlapping_rows_are_refused(no_launch, which):
    """An expanded tensor has a row pitch of 0, which the C ABI takes as contiguous: the
    call would read, or write, rows past the tensor's end."""
    bad = overlapping()[which]
    for kw in (dict(k=bad), dict(v=bad)):
        for call in calls(batch_of(), **kw):
            with pytest.raises(ValueError, match="overlap"):
                call()


def test_overlapping_table_is_refused(no_launch):
    row = torch.zeros(1, 3, dtype=torch.int32)
    for table in (row.expand(2, 3), torch.zeros(8, dtype=torch.int32).as_strided((2, 3), (2, 1)),
                  torch.zeros(1, 1, dtype=torch.int32).expand(2, 1)):
        for call in calls(batch_of(), table=on_device(table)):
            with pytest.raises(ValueError, match="overlap"):
                call()


def test_one_row_may_have_any_pitch(no_launch):
    """A single row, or a single sequence's table, has nothing to overlap with."""
    one = on_device(torch.zeros(1, 2, 64, dtype=torch.bfloat16).as_strided((1, 2, 64), (0, 64, 1)))
    table = on_device(torch.zeros(3, dtype=torch.int32).as_strided((1, 3), (0, 1)))
    for call in calls(batch_of(n=1, rows=1), k=one, v=one, table=table):
        with pytest.raises(AssertionError, match="launched"):
            call()


@pytest.mark.parametrize("window", [-1, 2 ** 31, 2 ** 32, 2 ** 32 + 5])
def test_window_out_of_range_is_refused(no_launch, window):
    """A window is 32 bits in the C ABI: 2^32 + 5 must not become 5."""
    a = batch_of()
    with pytest.raises(ValueError, match="window"):
        attention.ssd_attn_varlen_fwd(a["x"], None, a["x"], *a["cache"], a["qsl"], a["lens"], a["table"],
                                      softmax_scale=1.0, window=window, workspace=a["ws"])


def test_workspace_serves_every_smaller_call():
    """Of two calls' sizes of which none of the second is larger, the second needs no more:
    one workspace serves layers of different head counts."""
    ws = attention.ssd_attn_varlen_workspace_size
    sizes = [(total, batch, heads, kv_heads, dim)
             for total in (1, 100, 4096) for batch in (1, 64) for dim in (64, 128)
             for heads, kv_heads in ((1, 1), (32, 1), (32, 4), (32, 8), (32, 32), (128, 1), (256, 2),
                                     (24, 8), (24, 1))]
    need = {s: ws(*s) for s in sizes}
    assert all(need.values())
    for large in sizes:
        for small in sizes:
            if all(a <= b for a, b in zip(small, large)):
                assert need[small] <= need[large], (small, large)


@pytest.mark.parametrize("scale", [2.5e38, -3.4e38])
def test_softmax_scale_that_overflows_is_refused(scale):
    """Scores are in units of log2: a scale whose product with log2(e) is infinite is none."""
    import ctypes
    lib = attention._functions()
    p = ctypes.c_void_p(1 << 12)
    assert lib.attn(p, None, p, p, p, None, None, p, p, p, 10, 2, 4, 2, 64, 8, 16, 4, 4, 0, 0, 0, scale, 0,
                    p, 1 << 40, None, None) == 1


def test_workspace_size_of_unsupported_heads():
    """A number of kv heads that the calls refuse has no workspace."""
    ws = attention.ssd_attn_varlen_workspace_size
    assert ws(10, 2, 65535, 65535, 64) > 0
    assert ws(10, 2, 65536, 65536, 64) == 0


@pytest.mark.parametrize("name,make", [
    ("qsl", lambda: torch.zeros((), dtype=torch.int32)), ("qsl", lambda: torch.zeros(0, dtype=torch.int32)),
    ("qsl", lambda: torch.zeros(3, 1, dtype=torch.int32)), ("qsl", lambda: torch.zeros(2, dtype=torch.int32)),
    ("qsl", lambda: torch.zeros(3, dtype=torch.int64)), ("lens", lambda: torch.zeros((), dtype=torch.int32)),
    ("lens", lambda: torch.zeros(3, dtype=torch.int32)), ("lens", lambda: torch.zeros(4, dtype=torch.int32)[::2]),
    ("table", lambda: torch.zeros(2, dtype=torch.int32)), ("table", lambda: torch.zeros(3, 3, dtype=torch.int32)),
    ("table", lambda: torch.zeros((), dtype=torch.int32)), ("table", lambda: torch.zeros(3, 2, dtype=torch.int32).T)])
def test_shapes_of_the_batch_are_refused(no_launch, name, make):
    a = batch_of()
    a[name] = on_device(make())
    for call in calls(a):
        with pytest.raises(ValueError):
            call()
