"""What the Python binding of the layer operators refuses of CUDA tensors: nothing is
launched and nothing is written."""
from __future__ import annotations

import pytest
import torch

import mamba_ssd_chunked_varlen_gb300 as pkg

pytestmark = pytest.mark.gpu

ROWS, C, N, W = 6, 64, 16, 4
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def zeros(*shape, dtype=BF16, device="cuda"):
    return torch.zeros(shape, dtype=dtype, device=device)


def batch():
    return dict(query_start_loc=torch.tensor([0, 2, 6], dtype=I32, device="cuda"),
                has_initial_state=zeros(2, dtype=torch.bool),
                cache_indices=torch.tensor([0, 2], dtype=I32, device="cuda"))


def refused(call, args, change):
    """`change` makes a good call (which the test makes last) a bad one."""
    good = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in args.items()}
    with pytest.raises((ValueError, pkg.SSDError)):
        call(**(args | change))
    torch.cuda.synchronize()
    for k, v in good.items():
        if isinstance(v, torch.Tensor) and v.dtype != torch.uint8:
            assert torch.equal(args[k], v), k
    call(**args)
    torch.cuda.synchronize()


def transposed(*shape, dtype=BF16):
    return zeros(*shape[::-1], dtype=dtype).permute(*range(len(shape))[::-1])


COMMON = [
    ("x", lambda: zeros(ROWS, C, dtype=torch.float16)), ("x", lambda: zeros(ROWS, C, 1)),
    ("x", lambda: zeros(1, C).expand(ROWS, C)), ("x", lambda: transposed(ROWS, C)),
    ("x", lambda: zeros(ROWS, C, device="cpu")), ("x", lambda: zeros(ROWS + 1, C)),
    ("x", lambda: zeros(ROWS, C + 4)[:, :C]), ("x", lambda: zeros(ROWS, C + 8)[:, 4:C + 4]),
    ("y", lambda: zeros(ROWS, C, dtype=F32)), ("y", lambda: zeros(ROWS, C + 8)),
    ("y", lambda: zeros(ROWS, C, device="cpu")), ("y", lambda: zeros(1, C).expand(ROWS, C)),
    ("query_start_loc", lambda: zeros(3, dtype=torch.int64)), ("query_start_loc", lambda: zeros(1, 3, dtype=I32)),
    ("query_start_loc", lambda: zeros(0, dtype=I32)), ("query_start_loc", lambda: zeros(3, dtype=I32, device="cpu")),
    ("query_start_loc", lambda: zeros(6, dtype=I32)[::2]), ("query_start_loc", lambda: zeros(4, dtype=I32)),
    ("has_initial_state", lambda: zeros(2, dtype=I32)), ("has_initial_state", lambda: zeros(3, dtype=torch.bool)),
    ("has_initial_state", lambda: zeros(2, dtype=torch.bool, device="cpu")),
    ("cache_indices", lambda: zeros(2, dtype=torch.int64)), ("cache_indices", lambda: zeros(1, dtype=I32)),
    ("cache_indices", lambda: zeros(1, dtype=I32).expand(2)), ("cache_indices", lambda: zeros(2, dtype=I32, device="cpu")),
    ("errors", lambda: zeros(1, dtype=torch.int64)), ("errors", lambda: zeros(0, dtype=I32)),
    ("errors", lambda: zeros(1, dtype=I32, device="cpu")),
]
CONV = [
    ("weight", lambda: zeros(C, W)), ("weight", lambda: zeros(C, 5, dtype=F32)), ("weight", lambda: zeros(C * W, dtype=F32)),
    ("weight", lambda: transposed(C, W, dtype=F32)), ("weight", lambda: zeros(C, W, dtype=F32, device="cpu")),
    ("weight", lambda: zeros(C, 3, dtype=F32)), ("bias", lambda: zeros(C)), ("bias", lambda: zeros(C + 8, dtype=F32)),
    ("bias", lambda: zeros(2 * C, dtype=F32)[::2]), ("conv_pool", lambda: zeros(3, W, C)),
    ("conv_pool", lambda: zeros(W - 1, C)), ("conv_pool", lambda: zeros()), ("conv_pool", lambda: zeros(3, W - 1, C, dtype=F32)),
    ("conv_pool", lambda: zeros(3, W - 1, 2 * C)[:, :, :C]), ("conv_pool", lambda: zeros(3, W - 1, C, device="cpu")),
]
SCAN = [
    ("dt", lambda: zeros(ROWS, 4)), ("dt", lambda: zeros(ROWS, C, dtype=F32)), ("dt", lambda: zeros(ROWS, 1).expand(ROWS, C)),
    ("B", lambda: zeros(ROWS, 2 * N)), ("B", lambda: zeros(1, N).expand(ROWS, N)), ("C", lambda: zeros(ROWS - 1, N)),
    ("C", lambda: zeros(ROWS, N, dtype=F32)), ("z", lambda: zeros(ROWS, C, dtype=F32)), ("z", lambda: zeros(ROWS, 2 * C)),
    ("A", lambda: zeros(C, N)), ("A", lambda: zeros(C, 24, dtype=F32)), ("A", lambda: zeros(C, dtype=F32)),
    ("A", lambda: transposed(C, N, dtype=F32)), ("D", lambda: zeros(C)), ("D", lambda: zeros(1, dtype=F32).expand(C)),
    ("dt_bias", lambda: zeros(C, device="cpu", dtype=F32)), ("ssm_pool", lambda: zeros(3, C, N, dtype=torch.float16)),
    ("ssm_pool", lambda: zeros(3, N, C, dtype=F32)), ("ssm_pool", lambda: zeros(dtype=F32)),
    ("ssm_pool", lambda: zeros(C, N, dtype=F32)), ("ssm_pool", lambda: zeros(6, C, N, dtype=F32)[::2]),
    ("workspace", lambda: None), ("workspace", lambda: zeros(16, dtype=torch.uint8)),
    ("workspace", lambda: zeros(1 << 20, dtype=I32)), ("workspace", lambda: zeros(1 << 20, dtype=torch.uint8, device="cpu")),
    ("workspace", lambda: zeros((1 << 20) + 16, dtype=torch.uint8)[16:]),
]


@pytest.mark.parametrize("what", range(len(COMMON + CONV)))
def test_conv(what):
    name, make = (COMMON + CONV)[what]
    args = dict(y=zeros(ROWS, C), x=zeros(ROWS, C) + 1, weight=zeros(C, W, dtype=F32) + 1, bias=zeros(C, dtype=F32),
                conv_pool=zeros(3, W - 1, C), errors=zeros(1, dtype=I32)) | batch()
    refused(pkg.ssd_causal_conv_varlen_fwd, args, {name: make()})


@pytest.mark.parametrize("what", range(len(COMMON + SCAN)))
def test_scan(what):
    name, make = (COMMON + SCAN)[what]
    args = dict(y=zeros(ROWS, C), x=zeros(ROWS, C) + 1, dt=zeros(ROWS, C), A=zeros(C, N, dtype=F32) - 1,
                B=zeros(ROWS, N) + 1, C=zeros(ROWS, N) + 1, D=zeros(C, dtype=F32), z=zeros(ROWS, C) + 1,
                dt_bias=zeros(C, dtype=F32), ssm_pool=zeros(3, C, N, dtype=F32), errors=zeros(1, dtype=I32),
                workspace=pkg.alloc_selective_scan_workspace(ROWS, 2, C, N)) | batch()
    refused(pkg.ssd_selective_scan_varlen_fwd, args, {name: make()})


@pytest.mark.parametrize("name,make", [
    ("x", lambda: zeros(ROWS * C)), ("x", lambda: zeros(ROWS, C, dtype=F32)), ("x", lambda: zeros(1, C).expand(ROWS, C)),
    ("x", lambda: zeros(ROWS, C + 4)[:, :C]), ("x", lambda: zeros(ROWS, C, device="cpu")),
    ("y", lambda: zeros(ROWS, C, dtype=F32)), ("y", lambda: zeros(ROWS, C, dtype=torch.int8)),
    ("y", lambda: zeros(ROWS, 2 * C)), ("residual", lambda: zeros(ROWS, C, dtype=F32)),
    ("residual", lambda: zeros(1, C).expand(ROWS, C)), ("gate", lambda: zeros(ROWS, C)),
    ("weight", lambda: zeros(C)), ("weight", lambda: zeros(2 * C, dtype=F32)[::2]), ("weight", lambda: zeros(8, dtype=F32)),
    ("scale", lambda: zeros(ROWS, 1, dtype=F32)), ("ngroups", lambda: 3), ("ngroups", lambda: 0), ("ngroups", lambda: 16),
    ("eps", lambda: 0.0), ("eps", lambda: 2.0),
])
def test_norm(name, make):
    args = dict(y=zeros(ROWS, C), x=zeros(ROWS, C) + 1, weight=zeros(C, dtype=F32) + 1, residual=zeros(ROWS, C))
    refused(pkg.ssd_rms_norm_fwd, args, {name: make()})


def test_norm_codes():
    args = dict(y=zeros(ROWS, C, dtype=torch.int8), x=zeros(ROWS, C) + 1, weight=None, scale=zeros(ROWS, 2, dtype=F32),
                ngroups=2)
    for change in (dict(scale=None), dict(scale=zeros(ROWS, 1, dtype=F32)), dict(scale=zeros(ROWS, 2)),
                   dict(scale=zeros(ROWS, 4, dtype=F32)[:, ::2]), dict(y=zeros(ROWS, C)),
                   dict(y=zeros(ROWS, C, dtype=torch.uint8))):
        refused(pkg.ssd_rms_norm_fwd, args | dict(y=torch.zeros_like(args["y"]), scale=torch.zeros_like(args["scale"])),
                change)


ROPE = [
    ("q", lambda: None), ("q", lambda: zeros(ROWS, 4, 64, dtype=F32)), ("q", lambda: zeros(ROWS, 256)),
    ("q", lambda: zeros(ROWS, 4, 128)[..., :64]), ("q", lambda: zeros(1, 4, 64).expand(ROWS, 4, 64)),
    ("q_out", lambda: zeros(ROWS, 2, 64)), ("q_out", lambda: zeros(ROWS, 4, 64, device="cpu")),
    ("k", lambda: zeros(ROWS + 1, 2, 64)), ("k", lambda: zeros(ROWS, 2, 128)), ("k", lambda: zeros(ROWS, 2, 64, device="cpu")),
    ("table", lambda: zeros(32, dtype=F32)), ("table", lambda: zeros(1, 32, dtype=torch.int64)),
    ("table", lambda: zeros(12, dtype=torch.int64)), ("table", lambda: zeros(40, dtype=torch.int64)),
    ("table", lambda: zeros(64, dtype=torch.int64)[::2]), ("table", lambda: zeros(32, dtype=torch.int64, device="cpu")),
    ("query_start_loc", lambda: zeros(3, dtype=torch.int64)), ("query_start_loc", lambda: zeros(6, dtype=I32)[::2]),
    ("kv_lens", lambda: zeros(2, dtype=torch.int64)), ("kv_lens", lambda: zeros(3, dtype=I32)),
    ("kv_lens", lambda: zeros(2, dtype=I32, device="cpu")), ("magnitude", lambda: float("inf")),
    ("errors", lambda: zeros(1)),
]


@pytest.mark.parametrize("what", range(len(ROPE) + 2))
def test_rope(what):
    name, make = (ROPE + [("k_out", lambda: None), ("k_out", lambda: zeros(ROWS, 2, 64, dtype=F32))])[what]
    args = dict(q_out=zeros(ROWS, 4, 64), q=zeros(ROWS, 4, 64) + 1, k_out=zeros(ROWS, 2, 64), k=zeros(ROWS, 2, 64) + 1,
                table=pkg.alloc_rope_table(pkg.rope_frequencies(64)[0]), errors=zeros(1, dtype=I32),
                query_start_loc=batch()["query_start_loc"], kv_lens=zeros(2, dtype=I32) + 9)
    refused(pkg.ssd_rope_varlen_fwd, args, {name: make()})


WRITE = [
    ("v", lambda: zeros(ROWS, 4, 64)), ("v", lambda: zeros(ROWS, 2, 64, dtype=F32)), ("v", lambda: zeros(1, 2, 64).expand(ROWS, 2, 64)),
    ("k", lambda: zeros(ROWS, 4, 64)), ("k_scale", lambda: zeros(4, 2, 16, dtype=F32)),
    ("k_cache", lambda: zeros(4, 2, 16, 64, dtype=torch.int8)), ("k_cache", lambda: zeros(4, 2, 16, 64, device="cpu")),
    ("v_cache", lambda: zeros(4, 2, 8, 64)), ("block_table", lambda: zeros(2, 1, dtype=torch.int64)),
    ("block_table", lambda: zeros(3, 1, dtype=I32)),
]


@pytest.mark.parametrize("what", range(len(ROPE[1:] + WRITE)))
def test_rope_write(what):
    name, make = (ROPE[1:] + WRITE)[what]
    args = dict(q_out=zeros(ROWS, 4, 64), q=zeros(ROWS, 4, 64) + 1, k=zeros(ROWS, 2, 64) + 1, v=zeros(ROWS, 2, 64) + 1,
                table=pkg.alloc_rope_table(pkg.rope_frequencies(64)[0]), k_cache=zeros(4, 2, 16, 64),
                v_cache=zeros(4, 2, 16, 64), k_scale=None, v_scale=None, errors=zeros(1, dtype=I32),
                query_start_loc=batch()["query_start_loc"], kv_lens=zeros(2, dtype=I32) + 9,
                block_table=torch.tensor([[0], [3]], dtype=I32, device="cuda"))
    refused(pkg.ssd_rope_kv_cache_write, args, {name: make()})
