"""What is measured of the paged-cache operators, and their plain forms.

Two operators serve the attention layers of a hybrid model, beside its scan
layers and on the same ragged batch (query_start_loc):

  write / read   the new tokens' keys and values go into a paged cache (bf16, or
                 8-bit codes with one fp32 scale per token and head), and tokens
                 are read back from it
  attend         causal grouped-query attention of every sequence's new tokens
                 over its tokens in that cache

`prepare` makes what a serving loop has in hand before the call, `run` makes one
pass, `exact` gives the same answer in 64 bits.  The plain forms are elementary
torch operations in 32 bits on the batch padded to its longest sequence.

Definitions.  Sequence b has n_b = query_start_loc[b+1] - query_start_loc[b] new
tokens, the last n_b of its kv_lens[b] tokens; token j of a sequence lies in row
j % page of page block_table[b, j // page].  Caches are (pages, kv heads, page,
dim), scales (pages, kv heads, page).  A row x of `dim` elements is stored as
code = round(x * (M / a)) with a = max(|x|, 2^-60 at least) and M = 127 (int8) or
448 (fp8 e4m3, rounded to nearest even), its scale is a / M, and it stands for
code * scale.  The query at position i sees the keys j <= i, with a window w > 0
only those with j > i - w.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "int8": torch.int8}
TOP = {"fp8": 448.0, "int8": 127.0}
TINY = 2.0 ** -60

# the largest listed attention (elements of the padded score matrix) and cache
# (elements of one of K and V, padded): no drawn case goes beyond either
MOST_SCORES = 32 * 2048 * 32768
MOST_CACHE = 8 * 65536 * 8 * 128
MOST_ROWS = 16384 * 8 * 128


# ------------------------------------------------------------------ the cases

def _attend(name, kind, batch, new, kv, heads, kv_heads, dim, page, single=0, window=0, lse=False,
            lens=0):
    return {"name": name, "op": "attend", "type": kind, "batch": batch, "new_min": new[0],
            "new_max": new[1], "kv_min": kv[0], "kv_max": kv[1], "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "single": single, "window": window,
            "lse": lse, "lens": lens}


def _cache(name, op, kind, batch, new, kv, kv_heads, dim, page, single=0, lens=0):
    return {"name": name, "op": op, "type": kind, "batch": batch, "new_min": new[0],
            "new_max": new[1], "kv_min": kv[0], "kv_max": kv[1], "kv_heads": kv_heads, "dim": dim,
            "page": page, "single": single, "lens": lens}


def listed():
    return [
        # one user, one token, a short context: the smallest call, where latency counts
        _attend("decode_one", "bf16", 1, (1, 1), (777, 777), 32, 8, 128, 16),
        # a decode step of a busy server: ragged contexts, 8-bit cache
        _attend("decode_batch", "int8", 64, (1, 1), (1, 8192), 32, 8, 128, 16),
        # a few users with long documents: the whole step is reading the cache
        _attend("decode_long", "fp8", 8, (1, 1), (49001, 65535), 64, 8, 128, 64),
        # five proposed tokens a sequence are verified at once; three query heads a
        # kv head, narrow heads; the log-sum-exp joins the part of a shared prefix
        _attend("verify", "bf16", 32, (5, 5), (5, 4099), 24, 8, 64, 32, lse=True),
        # prompts' chunks and decoding sequences in one batch
        _attend("mixed", "int8", 24, (64, 500), (501, 4095), 16, 2, 128, 32, single=20),
        # a long document's chunk: the largest call, bound by the tensor cores
        _attend("chunk_long", "bf16", 1, (2048, 2048), (32768, 32768), 32, 8, 128, 128),
        # two prompts' chunks over an 8-bit cache; odd context lengths
        _attend("chunk_fp8", "fp8", 2, (1024, 1024), (12001, 16383), 32, 8, 128, 64),
        # prompts in layers with a sliding window, one query head a kv head
        _attend("window", "bf16", 4, (700, 1111), (1111, 5000), 16, 16, 64, 16, window=1024,
                lse=True),
        # a decode step's new rows into an 8-bit cache, and back
        _cache("write_decode", "write", "fp8", 64, (1, 1), (1, 8192), 8, 128, 16),
        # whole prompts into an 8-bit cache, and back
        _cache("write_prompt", "write", "int8", 8, (1, 4096), (4096, 4096), 8, 128, 64),
        # prompts into a bf16 cache
        _cache("write_plain", "write", "bf16", 8, (129, 2049), (2049, 4097), 8, 128, 16),
        # whole contexts read back, as to move them elsewhere
        _cache("read_context", "read", "int8", 16, (1, 8192), (8192, 8192), 8, 128, 32),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        kind = rng.choice(("bf16", "fp8", "int8"))
        dim = rng.choice((64, 128))
        page = rng.choice((16, 32, 64, 128))
        kv_heads = rng.choice((1, 2, 4, 8, 16))
        lens = rng.randrange(1 << 30)
        if rng.random() < 0.35:
            op = rng.choice(("write", "read"))
            batch = _log(rng, 1, 128)
            new = _log(rng, 1, 8192)
            kv = new if op == "read" else new + _log(rng, 1, 4096) - 1
            c = _cache("", op, kind, batch, (max(1, new // rng.choice((1, 3, 50))), new), (new, kv),
                       kv_heads, dim, page, single=rng.choice((0, batch // 2)), lens=lens)
            if batch * new * kv_heads * dim > MOST_ROWS or batch * kv * kv_heads * dim > MOST_CACHE // 4:
                continue
        else:
            group = rng.choice((1, 2, 3, 4, 5, 7, 8, 16))
            batch = _log(rng, 1, 128)
            new = 1 if rng.random() < 0.35 else _log(rng, 2, 2048)
            kv = new + _log(rng, 1, 65536) - 1
            c = _attend("", kind, batch, (max(1, new // rng.choice((1, 2, 20))), new),
                        (max(new, kv // rng.choice((1, 3, 100))), kv), kv_heads * group, kv_heads,
                        dim, page, single=rng.choice((0, 0, batch // 2, batch - 1)),
                        window=rng.choice((0, 0, _log(rng, 16, 4096))), lse=rng.random() < 0.5,
                        lens=lens)
            if (kv_heads * group > 64 or batch * kv * kv_heads * dim > MOST_CACHE
                    or batch * kv * kv_heads * group * new > MOST_SCORES):
                continue
        del c["name"]
        return c


def _lengths(case):
    """(new tokens, context length) of every sequence, from the case alone: the
    context counts the new tokens."""
    rng = random.Random("%d %d %d" % (case["lens"], case["batch"], case["kv_max"]))
    out = []
    for b in range(case["batch"]):
        new = 1 if b < case["single"] else rng.randint(case["new_min"], case["new_max"])
        kv = new if case["op"] == "read" else max(new, rng.randint(case["kv_min"], case["kv_max"]))
        out.append((new, kv))
    # (the sequences with one token are not the first ones of the batch)
    rng.shuffle(out)
    return out


def _visible(case, new, kv):
    """Pairs of query and key of one sequence, and the keys that any query sees."""
    w = case["window"] or kv
    first = kv - new
    pairs = sum(min(i + 1, w) for i in range(first, kv))
    return pairs, min(kv, new + w - 1)


def work(case):
    lens = _lengths(case)
    kh, d = case["kv_heads"], case["dim"]
    size = 2 if case["type"] == "bf16" else 1
    row = 2 * kh * (d * size + (0 if size == 2 else 4))      # K and V of one token, with scales
    tables = 8 * case["batch"] + 4 * sum(-(-kv // case["page"]) for _, kv in lens)
    total = sum(n for n, _ in lens)
    wide = total * 2 * kh * d * 2                             # K and V of the new tokens in bf16
    if case["op"] == "write":
        back = 0 if case["type"] == "bf16" else total * row + wide
        return {"bytes": wide + total * row + back + tables, "flops": 4 * total * kh * d}
    if case["op"] == "read":
        return {"bytes": wide + total * row + tables, "flops": 2 * total * kh * d}
    seen = [_visible(case, n, kv) for n, kv in lens]
    qo = 2 * total * case["heads"] * d * 2 + (4 * total * case["heads"] if case["lse"] else 0)
    return {"bytes": qo + sum(s for _, s in seen) * row + tables,
            "flops": 4 * d * case["heads"] * sum(p for p, _ in seen)}


# ------------------------------------------------------------------ the inputs

def _codes(x, kind):
    """Codes and scales of rows (the last axis), 32 bits until the code."""
    a = x.abs().amax(-1).clamp(min=TINY)
    top = torch.full_like(a, TOP[kind])   # (a quotient with a number would go by its reciprocal)
    y = x * (top / a).unsqueeze(-1)
    code = y.round().to(torch.int8) if kind == "int8" else y.to(torch.float8_e4m3fn)
    return code, a / top


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rng = random.Random(seed)
    lens = _lengths(case)
    batch, page, kh, d, kind = (case[k] for k in ("batch", "page", "kv_heads", "dim", "type"))
    total = sum(n for n, _ in lens)
    need = [-(-kv // page) for _, kv in lens]
    pages = sum(need) + 3
    order = list(range(pages))
    rng.shuffle(order)
    table = torch.zeros((batch, max(need)), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    start = torch.zeros(batch + 1, dtype=torch.int32)
    start[1:] = torch.tensor([n for n, _ in lens]).cumsum(0)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    # keys have a few channels that are larger than the others, and tokens differ in size
    channel = torch.ones(d, device=dev)
    channel[torch.randperm(d, generator=g, device=dev)[:max(1, d // 16)]] = 4.0

    def keys(*shape):
        return normal(*shape) * channel * torch.exp(0.3 * normal(*shape[:-1], 1))

    s = {"case": case, "max_new": max(n for n, _ in lens), "max_kv": max(kv for _, kv in lens),
         "total": total, "query_start_loc": start.to(dev), "block_table": table.to(dev),
         "kv_lens": torch.tensor([kv for _, kv in lens], dtype=torch.int32, device=dev),
         "k_scale": None, "v_scale": None}
    for name, rows in (("k", keys), ("v", normal)):
        x = rows(pages, kh, page, d)
        if kind == "bf16":
            s[name + "_cache"] = x.to(torch.bfloat16)
        else:
            s[name + "_cache"], s[name + "_scale"] = _codes(x.to(torch.bfloat16).float(), kind)
        del x
    if case["op"] == "write":
        s["k"] = keys(total, kh, d).to(torch.bfloat16)
        s["v"] = normal(total, kh, d).to(torch.bfloat16)
    if case["op"] == "attend":
        s["q"] = normal(total, case["heads"], d).to(torch.bfloat16)
        s["softmax_scale"] = 1.0 / math.sqrt(d)
    if own:   # the buffers that a serving loop keeps: the results' and the workspace
        import mamba_ssd_chunked_varlen_gb300 as pkg
        s["errors"] = torch.zeros(1, dtype=torch.int32, device=dev)
        if case["op"] == "attend":
            s["o"] = torch.empty((total, case["heads"], d), dtype=torch.bfloat16, device=dev)
            s["lse"] = (torch.empty((total, case["heads"]), dtype=torch.float32, device=dev)
                        if case["lse"] else None)
            s["workspace"] = pkg.alloc_attn_workspace(total, batch, case["heads"], kh, d)
        else:
            s["k_out"] = torch.empty((total, kh, d), dtype=torch.bfloat16, device=dev)
            s["v_out"] = torch.empty_like(s["k_out"])
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    if not own:
        return {"attend": _plain_attend, "write": _plain_write, "read": _plain_read}[case["op"]](s)
    import mamba_ssd_chunked_varlen_gb300 as pkg
    cache = (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    where = (s["query_start_loc"], s["kv_lens"], s["block_table"])
    if case["op"] == "attend":
        pkg.ssd_attn_varlen_fwd(s["o"], s["lse"], s["q"], *cache, *where,
                                softmax_scale=s["softmax_scale"], window=case["window"],
                                workspace=s["workspace"], errors=s["errors"])
        return {"o": s["o"], "lse": s["lse"]}
    if case["op"] == "write":
        pkg.ssd_kv_cache_write(s["k"], s["v"], *cache, *where, errors=s["errors"])
        if case["type"] == "bf16":
            return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    pkg.ssd_kv_cache_read(s["k_out"], s["v_out"], *cache, *where, errors=s["errors"])
    out = {"k": s["k_out"], "v": s["v_out"]}
    if case["op"] == "write":
        out |= {"k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    return out


# ------------------------------------------------------------------ the plain forms

def _new_rows(s):
    """Page and row in the page of every new token."""
    start = s["query_start_loc"].long()
    t = torch.arange(s["total"], device=start.device)
    b = torch.searchsorted(start, t, right=True) - 1
    at = s["kv_lens"].long()[b] - start[b + 1] + t
    page = s["case"]["page"]
    return s["block_table"].long()[b, at // page], at % page


def _plain_write(s):
    kind = s["case"]["type"]
    page, row = _new_rows(s)
    for name in ("k", "v"):
        if kind == "bf16":
            s[name + "_cache"][page, :, row] = s[name]
        else:
            code, scale = _codes(s[name].float(), kind)
            # (torch has no indexed store of fp8: its bytes are stored)
            s[name + "_cache"].view(torch.int8)[page, :, row] = code.view(torch.int8)
            s[name + "_scale"][page, :, row] = scale
    if kind == "bf16":
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    return _plain_read(s) | {"k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _plain_read(s):
    kind = s["case"]["type"]
    page, row = _new_rows(s)
    return {name: _rows(s, name, kind, page, row).to(torch.bfloat16) for name in ("k", "v")}


def _rows(s, name, kind, page, row):
    """The values of cache rows in 32 bits: page and row of any one shape, then (kv heads, dim)."""
    cache = s[name + "_cache"]
    if kind == "bf16":
        return cache[page, :, row].float()
    x = cache.view(torch.int8)[page, :, row].view(cache.dtype).float()
    return x * s[name + "_scale"][page, :, row].unsqueeze(-1)


def _plain_attend(s):
    case = s["case"]
    h, kh, d, page, w = (case[k] for k in ("heads", "kv_heads", "dim", "page", "window"))
    batch, new, kv, dev = case["batch"], s["max_new"], s["max_kv"], s["q"].device
    start, kv_lens = s["query_start_loc"].long(), s["kv_lens"].long()
    n = start[1:] - start[:-1]
    j = torch.arange(kv, device=dev)
    pages = s["block_table"].long()[:, j // page]
    rows = (j % page).expand(batch, kv)
    # (batch, kv heads, query rows of the group, keys)
    i = torch.arange(new, device=dev)
    q = s["q"].float()[(start[:-1, None] + i).clamp(max=s["total"] - 1)]
    q = q.view(batch, new, kh, h // kh, d).permute(0, 2, 1, 3, 4).reshape(batch, kh, -1, d)
    x = q @ _rows(s, "k", case["type"], pages, rows).permute(0, 2, 3, 1) * s["softmax_scale"]
    x = x.view(batch, kh, new, h // kh, kv)
    at = (kv_lens - n)[:, None] + i
    seen = (j <= at[..., None]) & (j < kv_lens[:, None, None])
    if w:
        seen &= j > at[..., None] - w
    x.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    del x
    total = p.sum(-1, keepdim=True)
    v = _rows(s, "v", case["type"], pages, rows).permute(0, 2, 1, 3)
    o = (p.view(batch, kh, -1, kv) @ v).view(batch, kh, new, h // kh, d)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).reshape(batch, new, h, d)
    t = torch.arange(s["total"], device=dev)
    b = torch.searchsorted(start, t, right=True) - 1
    out = {"o": o[b, t - start[b]].to(torch.bfloat16), "lse": None}
    if case["lse"]:
        lse = (top + torch.log(total)).permute(0, 2, 1, 3, 4).reshape(batch, new, h)
        out["lse"] = lse[b, t - start[b]]
    return out


# ------------------------------------------------------------------ in 64 bits

def _exact_codes(x, kind):
    """Codes (as numbers) and scales of rows, from the definition, in 64 bits."""
    a = torch.maximum(x.abs().amax(-1), torch.tensor(TINY, dtype=x.dtype, device=x.device))
    y = x * (TOP[kind] / a)[..., None]
    if kind == "int8":
        return torch.round(y), a / TOP[kind]
    # e4m3: three bits after the leading one, exponents from -6 on
    _, e = torch.frexp(y)
    step = torch.ldexp(torch.ones_like(y), (e - 1).clamp(min=-6) - 3)
    return torch.round(y / step) * step, a / TOP[kind]


def exact(case, seed):
    lens = _lengths(case)
    if case["op"] == "attend":
        flops = 4 * case["dim"] * case["heads"] * sum(n * kv for n, kv in lens)
        if flops > 4e12:   # over about 20 s in 64 bits
            return None
    s = prepare(case, seed)
    page, kind = case["page"], case["type"]
    start = s["query_start_loc"].tolist()

    def rows(b, j):
        return s["block_table"][b].long()[j // page], j % page

    def stored(name, b, j):
        p, r = rows(b, j)
        x = s[name + "_cache"].view(torch.int8 if kind != "bf16" else torch.bfloat16)
        x = x[p, :, r].view(TYPES[kind])
        x = x.float().double()
        return x if kind == "bf16" else x * s[name + "_scale"][p, :, r].double()[..., None]

    if case["op"] == "write":
        out = {}
        for name in ("k", "v"):
            x = s[name].double()
            back = torch.empty_like(x)
            cache = s[name + "_cache"].double() if kind == "bf16" else None
            scales = None if kind == "bf16" else s[name + "_scale"].double()
            for b, (n, kv) in enumerate(lens):
                p, r = rows(b, torch.arange(kv - n, kv, device=x.device))
                mine = slice(start[b], start[b + 1])
                if kind == "bf16":
                    cache[p, :, r] = x[mine]
                else:
                    code, scale = _exact_codes(x[mine], kind)
                    back[mine] = code * scale[..., None]
                    scales[p, :, r] = scale
            if kind == "bf16":
                out[name + "_cache"] = cache
            else:
                out[name], out[name + "_scale"] = back, scales
        return out
    if case["op"] == "read":
        return {name: torch.cat([stored(name, b, torch.arange(kv - n, kv, device="cuda"))
                                 for b, (n, kv) in enumerate(lens)]) for name in ("k", "v")}
    o, lse = [], []
    group = case["heads"] // case["kv_heads"]
    for b, (n, kv) in enumerate(lens):
        j = torch.arange(kv, device="cuda")
        k, v = (stored(name, b, j).transpose(0, 1) for name in ("k", "v"))     # (kv heads, keys, dim)
        q = s["q"][start[b]:start[b + 1]].double()
        q = q.unflatten(1, (case["kv_heads"], group)).permute(1, 2, 0, 3)      # (kv heads, group, new, dim)
        x = torch.einsum("hgnd,hkd->hgnk", q, k) * s["softmax_scale"]
        i = torch.arange(kv - n, kv, device="cuda")[:, None]
        hidden = (j > i) | ((j <= i - case["window"]) if case["window"] else (j < 0))
        x[:, :, hidden] = -math.inf
        z = torch.logsumexp(x, -1)
        o.append(torch.einsum("hgnk,hkd->nhgd", torch.exp(x - z[..., None]), v).flatten(1, 2))
        lse.append(z.permute(2, 0, 1).flatten(1, 2))
    return {"o": torch.cat(o), "lse": torch.cat(lse) if case["lse"] else None}
