"""Shared helpers of the paged-cache tests: a ragged batch with its cache, and
the 64-bit answers on the CPU.

Error bounds (u = 2^-8 is bf16's relative rounding: 8 significant bits).  A probability enters the
product with v rounded to bf16 (relative error u) and the result is rounded to
bf16 once (u of |o| <= sum p|v|); a score is a sum of head_dim products in fp32,
so it is off by at most eps = head_dim 2^-23 scale max sum|q k|, which changes
a normalised probability by a factor of at most e^(2 eps); the exponentials'
own error (2^-20 covers it) and the fp32 sums over n keys (n 2^-24 each in l and
in o) come on top, and a probability below fp32's normal numbers counts as zero:

    |o - o_ref| <= (2 u (1 + 2^-6) + 2 eps + 2^-20 + 2 n 2^-24) sum_j p_j |v_j|
                   + 2^-126 sum_j |v_j|
    |lse - lse_ref| <= eps + 2^-20 + n 2^-24 + 2^-22 |lse_ref|
"""
from __future__ import annotations

import math

import numpy as np

TOP = {"int8": 127.0, "fp8": 448.0}
TINY = 2.0 ** -60


def torch_type(kind):
    import torch
    return {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "int8": torch.int8}[kind]


class Batch:
    """Ragged batch on `device`: lens is [(new rows, kv_len)].  Cache rows that
    no sequence owns hold NaN (or NaN scales), table entries past a sequence's
    last page an index that is out of range."""

    def __init__(self, lens, heads, kv_heads, dim, page, kind, seed=0, device="cuda",
                 q_scale=1.0, spare=2):
        import torch
        g = torch.Generator().manual_seed(seed)
        self.lens, self.heads, self.kv_heads, self.dim = lens, heads, kv_heads, dim
        self.page, self.kind, self.device = page, kind, device
        batch = len(lens)
        self.total = sum(n for n, _ in lens)
        need = [-(-kv // page) for _, kv in lens]
        self.pages = sum(need) + spare
        order = torch.randperm(self.pages, generator=g).tolist()
        width = max(need + [1]) + 1
        table = torch.full((batch, width), 1 << 30, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        qsl = torch.zeros(batch + 1, dtype=torch.int32)
        if batch:
            qsl[1:] = torch.tensor([n for n, _ in lens]).cumsum(0)
        self.table_cpu = table
        self.query_start_loc = qsl.to(device)
        self.kv_lens = torch.tensor([kv for _, kv in lens], dtype=torch.int32).to(device)
        self.block_table = table.to(device)
        shape = (self.pages, kv_heads, page, dim)
        # every sequence's keys and values, exact bf16 numbers
        self.k_seq = [torch.randn((kv, kv_heads, dim), generator=g).bfloat16() for _, kv in lens]
        self.v_seq = [torch.randn((kv, kv_heads, dim), generator=g).bfloat16() for _, kv in lens]
        self.q = (torch.randn((self.total, heads, dim), generator=g) * q_scale).bfloat16().to(device)
        self.k_scale = self.v_scale = None
        if kind == "bf16":
            self.k_cache = torch.full(shape, float("nan"), dtype=torch.bfloat16, device=device)
            self.v_cache = self.k_cache.clone()
        else:
            # (0x7f is NaN in e4m3)
            self.k_cache = torch.full(shape, 0x7f, dtype=torch.int8, device=device).view(torch_type(kind))
            self.v_cache = self.k_cache.clone()
            self.k_scale = torch.full(shape[:3], float("nan"), device=device)
            self.v_scale = self.k_scale.clone()
        self.errors = torch.zeros(1, dtype=torch.int32, device=device)

    @property
    def cache(self):
        return self.k_cache, self.v_cache, self.k_scale, self.v_scale

    @property
    def where(self):
        return self.query_start_loc, self.kv_lens, self.block_table

    def row_of(self, b, j):
        return int(self.table_cpu[b, j // self.page]), j % self.page

    def whole(self):
        """query_start_loc of the whole contexts (the running sum of kv_lens)."""
        import torch
        q = torch.zeros(len(self.lens) + 1, dtype=torch.int32)
        q[1:] = torch.tensor([kv for _, kv in self.lens]).cumsum(0)
        return q.to(self.device)

    def fill(self):
        """Write every sequence's whole context through ssd_kv_cache_write."""
        import torch
        import mamba_ssd_chunked_varlen_gb300 as pkg
        if sum(kv for _, kv in self.lens):
            pkg.ssd_kv_cache_write(torch.cat(self.k_seq).to(self.device),
                                   torch.cat(self.v_seq).to(self.device), *self.cache,
                                   self.whole(), self.kv_lens, self.block_table, errors=self.errors)
        return self

    def stored(self):
        """What the cache holds for every sequence, in 64 bits on the CPU: codes
        times scales as the cache has them (not as they ought to be)."""
        import torch
        out = []
        for name in ("k", "v"):
            cache, scale = getattr(self, name + "_cache"), getattr(self, name + "_scale")
            c = cache.float().cpu().double()
            if scale is not None:
                c = c * scale.cpu().double()[..., None]
            seqs = []
            for b, (_, kv) in enumerate(self.lens):
                j = torch.arange(kv)
                pages = self.table_cpu[b].long()[j // self.page]
                seqs.append(c[pages, :, j % self.page].numpy())
            out.append(seqs)
        return out

    def attend(self, softmax_scale=None, window=0, lse=True, stream=None, workspace=None):
        import torch
        import mamba_ssd_chunked_varlen_gb300 as pkg
        scale = 1 / math.sqrt(self.dim) if softmax_scale is None else softmax_scale
        o = torch.full_like(self.q, float("nan"))
        z = torch.full((self.total, self.heads), float("nan"), device=self.device) if lse else None
        if workspace is None:
            workspace = pkg.alloc_attn_workspace(self.total, len(self.lens), self.heads,
                                                 self.kv_heads, self.dim)
        pkg.ssd_attn_varlen_fwd(o, z, self.q, *self.cache, *self.where, softmax_scale=scale,
                                window=window, workspace=workspace, errors=self.errors, stream=stream)
        return o, z


def attend_ref(q, k, v, n, kv, scale, window):
    """One sequence in 64 bits: q (n, heads, dim), k and v (kv, kv heads, dim).
    Returns o, lse and the bounds of the module docstring."""
    heads, dim = q.shape[1], q.shape[2]
    kv_heads = k.shape[1]
    group = heads // kv_heads
    o = np.zeros((n, heads, dim))
    lse = np.full((n, heads), -np.inf)
    ob, lb = np.zeros((n, heads, dim)), np.zeros((n, heads))
    for h in range(heads):
        kh, vh = k[:, h // group], v[:, h // group]
        for i in range(n):
            at = kv - n + i
            lo, hi = max(0, at - window + 1) if window else 0, at + 1
            if hi <= lo:
                continue
            kk, vv = kh[lo:hi], vh[lo:hi]
            s = kk @ q[i, h] * scale
            eps = dim * 2.0 ** -23 * abs(scale) * np.max(np.abs(kk) @ np.abs(q[i, h]))
            m = s.max()
            p = np.exp(s - m)
            l = p.sum()
            o[i, h] = p @ vv / l
            lse[i, h] = m + np.log(l)
            ob[i, h] = (2 * 2.0 ** -8 * (1 + 2.0 ** -6) + 2 * eps + 2.0 ** -20
                        + 2 * (hi - lo) * 2.0 ** -24) * (p @ np.abs(vv) / l) \
                + 2.0 ** -126 * np.abs(vv).sum(0)
            lb[i, h] = eps + 2.0 ** -20 + (hi - lo) * 2.0 ** -24 + 2.0 ** -22 * abs(lse[i, h])
    return o, lse, ob, lb


def check_attend(batch: Batch, o, lse, softmax_scale=None, window=0, what="", stored=None):
    scale = 1 / math.sqrt(batch.dim) if softmax_scale is None else softmax_scale
    ks, vs = batch.stored() if stored is None else stored
    o, q = o.float().cpu().double().numpy(), batch.q.float().cpu().double().numpy()
    lse = None if lse is None else lse.cpu().double().numpy()
    at, worst = 0, 0.0
    for b, (n, kv) in enumerate(batch.lens):
        ro, rl, ob, lb = attend_ref(q[at:at + n], ks[b], vs[b], n, kv, scale, window)
        d = np.abs(o[at:at + n] - ro)
        assert np.all(d <= ob), f"{what} sequence {b} {(n, kv)}: o off by {np.nanmax(d):.3e}, " \
            f"{np.nanmax(d / np.maximum(ob, 1e-30)):.2f} of the bound, " \
            f"{np.isnan(d).sum()} NaN, {(~(d <= ob)).sum()} of {d.size}"
        worst = max(worst, float(np.max(d / np.maximum(ob, 1e-30), initial=0.0)))
        if lse is not None:
            empty = np.isinf(rl)
            got = lse[at:at + n]
            assert np.array_equal(np.isneginf(got), empty), f"{what} sequence {b}: empty rows"
            d = np.abs(np.where(empty, 0, got) - np.where(empty, 0, rl))
            assert np.all(d <= lb), f"{what} sequence {b}: lse off by {d.max():.3e}"
        at += n
    return worst
