"""The layer operators one after the other, as a model's layers run them: norm, convolution,
selective scan, gated norm and the rotated cache write and attention on one ragged batch,
step after step, prompts and single tokens; eagerly against each operator's formula in 64 bits
on what it was given, and as one captured graph against the eager calls, bit for bit."""
from __future__ import annotations

import os
import sys

import numpy as np
import pytest

from attn_helpers import Batch
from layer_helpers import U, Ragged, f64, near, same_bits
from test_causal_conv_gpu import conv_ref
from test_rms_norm_gpu import norm_ref
from test_selective_scan_gpu import scan_ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

CHANNELS, STATES, WIDTH, GROUPS, EPS = 264, 16, 4, 3, 1e-5


class Layer:
    """Norm of a residual stream, convolution of a column slice, scan, gated norm."""

    def __init__(self, slots, seed=0):
        import torch
        g = torch.Generator().manual_seed(seed)

        def normal(*shape):
            return torch.randn(shape, generator=g)

        self.norm1, self.norm2 = (1 + 0.2 * normal(2 * CHANNELS)).cuda(), (1 + 0.2 * normal(CHANNELS)).cuda()
        self.weight, self.bias = normal(CHANNELS, WIDTH).cuda(), normal(CHANNELS).cuda()
        self.A = -(torch.rand(CHANNELS, STATES, generator=g) * STATES + 0.5).cuda()
        self.D, self.dt_bias = normal(CHANNELS).cuda(), (normal(CHANNELS) - 3).cuda()
        self.conv_pool = torch.zeros(slots, WIDTH - 1, CHANNELS, dtype=torch.bfloat16, device="cuda")
        self.ssm_pool = torch.zeros(slots, CHANNELS, STATES, device="cuda")
        self.errors = torch.zeros(1, dtype=torch.int32, device="cuda")

    def buffers(self, rows):
        import torch
        bf = dict(dtype=torch.bfloat16, device="cuda")
        return dict(normed=torch.empty(rows, 2 * CHANNELS, **bf), mixed=torch.empty(rows, CHANNELS, **bf),
                    y=torch.empty(rows, CHANNELS, **bf),
                    codes=torch.empty(rows, CHANNELS, dtype=torch.int8, device="cuda"),
                    scale=torch.empty(rows, GROUPS, device="cuda"))

    def inputs(self, rows, seed):
        import torch
        g = torch.Generator().manual_seed(seed)
        shapes = dict(x=2 * CHANNELS, residual=2 * CHANNELS, dt=CHANNELS, B=STATES, C=STATES)
        return {k: torch.randn(rows, n, generator=g).bfloat16().cuda() for k, n in shapes.items()}

    def run(self, b, i, where, workspace):
        import mamba_ssd_chunked_varlen_gb300 as pkg
        pkg.ssd_rms_norm_fwd(b["normed"], i["x"], self.norm1, residual=i["residual"], eps=EPS)
        gate, x = b["normed"][:, :CHANNELS], b["normed"][:, CHANNELS:]
        pkg.ssd_causal_conv_varlen_fwd(b["mixed"], x, self.weight, self.bias, self.conv_pool, *where,
                                       errors=self.errors)
        pkg.ssd_selective_scan_varlen_fwd(b["y"], b["mixed"], i["dt"], self.A, i["B"], i["C"], self.D, None,
                                          self.dt_bias, self.ssm_pool, *where, workspace=workspace,
                                          errors=self.errors)
        pkg.ssd_rms_norm_fwd(b["codes"], b["y"], self.norm2, gate=gate, scale=b["scale"], ngroups=GROUPS, eps=EPS)


def check_step(layer, b, i, before, r, pools):
    """Every operator's output against its formula on the inputs that it had."""
    s, want, rel = norm_ref(f64(i["x"]), f64(layer.norm1), f64(before), None, 1, EPS)
    assert same_bits(i["residual"], (i["x"].float() + before.float()).bfloat16())
    near(f64(b["normed"]), want, np.abs(want) * (U + rel * (1 + U)), "norm")
    x = f64(b["normed"])[:, CHANNELS:]
    want, bound, pool = conv_ref(r, x, f64(layer.weight), f64(layer.bias), f64(pools[0]), True)
    near(f64(b["mixed"]), want, bound, "convolution")
    assert np.array_equal(f64(layer.conv_pool), pool)
    v = dict(x=f64(b["mixed"]), dt=f64(i["dt"]), A=f64(layer.A), B=f64(i["B"]), C=f64(i["C"]), D=f64(layer.D),
             z=None, dt_bias=f64(layer.dt_bias))
    want, bound, pool, off = scan_ref(r, v, f64(pools[1]), True, False)
    near(f64(b["y"]), want, bound, "scan")
    near(f64(layer.ssm_pool), pool, off, "states")
    _, want, rel = norm_ref(f64(b["y"]), f64(layer.norm2), None, f64(b["normed"])[:, :CHANNELS], GROUPS, EPS)
    scale = f64(b["scale"]).repeat(CHANNELS // GROUPS, 1)
    near(f64(b["codes"]) * scale, want, 0.5 * scale * (1 + 2.0 ** -6) + 2 * rel * np.abs(want), "gated norm")


def test_steps():
    """Prompts, their continuation and single tokens, slots carried along."""
    import mamba_ssd_chunked_varlen_gb300 as pkg
    import torch
    layer, seen = Layer(7), set()
    for step, lens in enumerate(([200, 3, 1], [1, 1, 1], [1, 150, 2, 0], [1, 1, 1, 1], [40, 1, 1, 1])):
        r = Ragged(lens, seed=0)
        r.slot[:] = np.arange(len(lens)) + 1
        r.has[:] = [int(s) in seen for s in r.slot]
        seen |= set(int(s) for s in r.slot)
        r.cache_indices.copy_(torch.tensor(r.slot))
        r.has_initial_state.copy_(torch.tensor(r.has))
        b, i = layer.buffers(r.rows), layer.inputs(r.rows, step)
        before, pools = i["residual"].clone(), (layer.conv_pool.clone(), layer.ssm_pool.clone())
        layer.run(b, i, r.where, pkg.alloc_selective_scan_workspace(r.rows, len(lens), CHANNELS, STATES))
        check_step(layer, b, i, before, r, pools)
        assert not layer.conv_pool[5:].any() and not layer.ssm_pool[5:].any()
    assert layer.errors.item() == 0


@pytest.mark.parametrize("lens", [[1] * 5, [300, 1, 1, 20, 0]])
def test_captured(lens):
    """A step with the cache write and the attention as one graph, replayed with new inputs
    and states, on a stream beside another call's."""
    import mamba_ssd_chunked_varlen_gb300 as pkg
    import torch
    r = Ragged(lens, seed=1)
    layer = Layer(r.slots, 1)
    ctx = Batch([(n, n + 37) for n in lens], 8, 2, 64, 16, "int8", seed=2).fill()
    table = pkg.alloc_rope_table(pkg.rope_frequencies(64)[0])
    ws = pkg.alloc_selective_scan_workspace(r.rows, len(lens), CHANNELS, STATES)
    attn_ws = pkg.alloc_attn_workspace(r.rows, len(lens), 8, 2, 64)
    b, i = layer.buffers(r.rows), layer.inputs(r.rows, 0)
    kv = torch.randn(2, r.rows, 2, 64, device="cuda").bfloat16()

    def step(b, q, o):
        layer.run(b, i, r.where, ws)
        pkg.ssd_rope_kv_cache_write(q, ctx.q, kv[0], kv[1], table, *ctx.cache, *ctx.where, errors=layer.errors)
        pkg.ssd_attn_varlen_fwd(o, None, q, *ctx.cache, *ctx.where, softmax_scale=0.125, workspace=attn_ws,
                                errors=layer.errors)

    state = layer.conv_pool, layer.ssm_pool, i["residual"], ctx.k_cache, ctx.v_cache, ctx.k_scale, ctx.v_scale
    q, o = torch.empty_like(ctx.q), torch.empty_like(ctx.q)
    kept = [t.clone() for t in state]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b, q, o)
    for t, k in zip(state, kept):
        t.copy_(k)
    for seed in range(3):
        for k, v in layer.inputs(r.rows, 10 + seed).items():
            if k != "residual":
                i[k].copy_(v)
        kv.normal_()
        before = [t.clone() for t in state]
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*b.values(), q, o, *state)]
        for t, k in zip(state, before):
            t.copy_(k)
        step(b, q, o)
        torch.cuda.synchronize()
        for x, y in zip(got, (*b.values(), q, o, *state)):
            assert same_bits(x, y)
    assert layer.errors.item() == 0


@pytest.mark.parametrize("scan", ["ssd", "selective"])
@pytest.mark.parametrize("cache", ["bfloat16", "int8"])
def test_example(scan, cache):
    """The serving example with either scan: no device-side errors, finite outputs, and the
    same bits again."""
    import torch
    import hybrid_serving as E
    outs = []
    for _ in range(2):
        block = E.HybridBlock(cache=getattr(torch, cache), scan=scan)
        outs.append([out for _, out in E.serve(block, 7)])
        assert block.flags() == 0
    for x, y in zip(*outs):
        assert torch.isfinite(x).all() and same_bits(x, y)


def test_two_streams():
    """Two layers with buffers, pools and workspaces of their own at once: the bits of one
    after the other."""
    import mamba_ssd_chunked_varlen_gb300 as pkg
    import torch
    r = [Ragged([700, 1, 40], seed=3), Ragged([1] * 64, seed=4)]
    got = []
    for together in (False, True):
        layers = [Layer(x.slots, 5 + k) for k, x in enumerate(r)]
        b = [layers[k].buffers(x.rows) for k, x in enumerate(r)]
        i = [layers[k].inputs(x.rows, k) for k, x in enumerate(r)]
        ws = [pkg.alloc_selective_scan_workspace(x.rows, len(x.lens), CHANNELS, STATES) for x in r]
        streams = [torch.cuda.Stream() for _ in r] if together else [torch.cuda.current_stream()] * 2
        torch.cuda.synchronize()
        for _ in range(5):
            for k, x in enumerate(r):
                with torch.cuda.stream(streams[k]):
                    layers[k].run(b[k], i[k], x.where, ws[k])
        torch.cuda.synchronize()
        got.append([t.clone() for k in range(2) for t in (*b[k].values(), layers[k].conv_pool, layers[k].ssm_pool,
                                                          i[k]["residual"])])
    for x, y in zip(*got):
        assert same_bits(x, y)
