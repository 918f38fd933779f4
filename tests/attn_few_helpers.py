"""The bound of the attention kernel of few rows (at most 16 query rows a kv head), tighter than
attn_helpers' by one rounding: a weight p (times its value's scale) enters the product with
v as two bf16, top = bf16(p) and rest = bf16(p - top), so that |p - top - rest| <= u |rest's
argument| <= u^2 p (u = 2^-8), 2^-15 with room; top v and rest v are two products a key, summed
in fp32 by the tensor cores, whose sums may be cut instead of rounded (2^-23 each):

    |o - o_ref| <= (u (1 + 2^-6) + 2^-15 + 2 eps + 2^-20 + 6 n 2^-24) sum_j p_j |v_j|
                   + 2^-126 sum_j |v_j|
"""
from __future__ import annotations

import numpy as np

from attn_helpers import attend_ref

U = 2.0 ** -8


def few_ref(q, k, v, n, kv, scale, window):
    """One sequence in 64 bits: o and its bound."""
    o, _, wide, _ = attend_ref(q, k, v, n, kv, scale, window)
    s = attend_ref(q, k, np.abs(v), n, kv, scale, window)[0]
    at = np.maximum(np.arange(kv - n, kv) + 1, 0)
    keys = (np.minimum(at, window) if window else at)[:, None, None]
    return o, wide - (U * (1 + 2.0 ** -6) - 2.0 ** -15 - 4 * keys * 2.0 ** -24) * s


def bf16(x):
    """fp32 numbers rounded to bf16 (nearest even), as fp32."""
    b = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7fff + (b >> 16 & 1)) & 0xffff0000
    return b.astype(np.uint32).view(np.float32)


def few_model(q, k, v, n, kv, scale, parts):
    """What a kernel with `parts` bf16 per weight gives (no window), sums in 64 bits."""
    heads, group = q.shape[1], q.shape[1] // k.shape[1]
    o = np.zeros(q.shape)
    for h in range(heads):
        for i in range(n):
            hi = kv - n + i + 1
            s = k[:hi, h // group] @ q[i, h] * scale
            p = np.exp(s - s.max()).astype(np.float32)
            w = bf16(p).astype(np.float64)
            if parts == 2:
                w = w + bf16(p - bf16(p))
            o[i, h] = w @ v[:hi, h // group] / p.astype(np.float64).sum()
    return bf16(o.astype(np.float32)).astype(np.float64)
