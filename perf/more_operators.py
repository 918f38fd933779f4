"""What is measured of the operators around the scan and the attention, and their
plain forms.

Four operators of a hybrid model's layers, on the ragged batch of the scan and the
attention (query_start_loc):

  conv   a short causal convolution of every channel, whose last inputs are kept
         in a pool of slots: y[t] = act(bias + sum_j w[j] x[t - (W-1) + j])
  scan   the selective scan whose step and decay are each channel's own:
         d = softplus(dt + dt_bias),  h = exp(d A) h + d x B,
         y = (C . h + D x) silu(z), the states in a pool of slots
  norm   root-mean-square norm of s = x + residual (the sum is written back) or
         s = x silu(gate), over groups of columns: y = s / sqrt(mean s^2 + eps) w,
         in bf16 or in 8-bit codes with a scale for each group of a row
  rope   rotary positions of q and k, alone or with the write of k and v into the
         paged cache: pairs (a, b) become (a cos - b sin, b cos + a sin) m at the
         angle position * frequency, pairs of neighbours or of half a head apart

`prepare` makes what a serving loop has in hand before the call, `run` makes one
pass, `exact` gives the same answer in 64 bits.  The plain forms are elementary
torch operations in 32 bits (angles in 64); the scan's doubles its steps log2(length)
times over all tokens at once.

8-bit rows: code = round(y * (M / a)) with a = max(|y|, 2^-60 at least) over the
group and M = 127 (int8) or 448 (fp8 e4m3, rounded to nearest even), the scale is
a / M.  They are returned as the values that they stand for, code * scale in bf16.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "int8": torch.int8, "fp32": torch.float32}
TOP = {"fp8": 448.0, "int8": 127.0}
TINY = 2.0 ** -60
EPS = 1e-5

# the largest listed cases: no drawn case goes beyond them
MOST_CONV = 25000 * 10240           # values
MOST_SCAN = 11000 * 8192 * 16       # states passed through
MOST_NORM = 8191 * 8192             # values
MOST_ROPE = 12000 * 48 * 128        # values rotated or written
MOST_CACHE = 4 * 40000 * 8 * 128    # elements of one of K and V


# ------------------------------------------------------------------ the cases

def _batch(batch, new, single=0, lens=0):
    return {"batch": batch, "new_min": new[0], "new_max": new[1], "single": single, "lens": lens}


def _conv(name, batch, channels, width=4, silu=True, bias=True):
    return {"name": name, "op": "conv", "channels": channels, "width": width, "silu": silu,
            "bias": bias, **batch}


def _scan(name, batch, channels, states, pool="fp32", gate=True):
    return {"name": name, "op": "scan", "channels": channels, "states": states, "pool": pool,
            "gate": gate, **batch}


def _norm(name, rows, dim, kind, groups=1, gate=False):
    return {"name": name, "op": "norm", "rows": rows, "dim": dim, "type": kind, "groups": groups,
            "gate": gate}


def _rope(name, batch, kv, kind, heads, kv_heads, dim, part, page=0, pairs="half", scaling="none"):
    """`kind` "none": q and k are rotated and not written; `part`: the rotated part of the head."""
    return {"name": name, "op": "rope", "type": kind, "kv_min": kv[0], "kv_max": kv[1], "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "part": part, "page": page, "pairs": pairs,
            "scaling": scaling, **batch}


def listed():
    return [
        # one decode step of a few users: the smallest call, where latency counts
        _conv("conv_step", _batch(8, (1, 1)), 4352),
        # a serving step, prompts' parts and single tokens mixed
        _conv("conv_mixed", _batch(256, (1, 127), 100), 4352),
        # whole prompts of a wide model
        _conv("conv_prompt", _batch(4, (4097, 8191)), 10240),
        # one decode step: the whole call is reading and writing the states
        _scan("scan_step", _batch(96, (1, 1)), 8192, 16),
        # a serving step: four prompts' parts and single tokens; half as many states again
        _scan("scan_mixed", _batch(24, (64, 900), 20), 4096, 16),
        # two long prompts of a wide model: the largest call, bound by the exponentials
        _scan("scan_prompt", _batch(2, (4097, 5500)), 8192, 16),
        # one decode step's rows for an 8-bit product
        _norm("norm_step", 48, 4096, "fp8"),
        # a serving step's rows for an 8-bit product, an odd number of them
        _norm("norm_codes", 4093, 5120, "int8"),
        # the gated norm behind the scan of whole prompts, eight groups
        _norm("norm_gated", 8191, 8192, "bf16", 8, True),
        # one decode step over an 8-bit cache
        _rope("rope_step", _batch(64, (1, 1)), (1, 8192), "fp8", 32, 8, 128, 128, 16),
        # parts of long documents, frequencies stretched for long contexts
        _rope("rope_prompt", _batch(4, (1000, 2999)), (9000, 40000), "int8", 32, 8, 128, 128, 64,
              scaling="ramp"),
        # half of each head in pairs of neighbours, positions far out, no cache
        _rope("rope_plain", _batch(3, (1500, 4000)), (100000, 1000000), "none", 16, 16, 64, 32,
              pairs="neighbours", scaling="linear"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_batch(rng, most):
    batch = _log(rng, 1, 256)
    top = 1 if rng.random() < 0.3 else _log(rng, 2, most)
    return _batch(batch, (max(1, top // rng.choice((1, 3, 30))), top), rng.choice((0, 0, batch // 2)),
                  rng.randrange(1 << 30))


def draw(rng):
    while True:
        op = rng.choice(("conv", "scan", "norm", "rope"))
        if op == "conv":
            c = _conv("", _draw_batch(rng, 8192), 8 * _log(rng, 16, 1280), rng.choice((2, 3, 4, 4)),
                      rng.random() < 0.8, rng.random() < 0.8)
            if sum(_lengths(c)) * c["channels"] > MOST_CONV:
                continue
        elif op == "scan":
            c = _scan("", _draw_batch(rng, 8192), 8 * _log(rng, 16, 1024), rng.choice((8, 16, 16, 32, 64)),
                      rng.choice(("fp32", "fp32", "bf16")), rng.random() < 0.7)
            work = max(sum(_lengths(c)), c["batch"]) * c["channels"] * c["states"]
            if work > MOST_SCAN // 4:
                continue
        elif op == "norm":
            gate = rng.random() < 0.4
            groups = rng.choice((1, 2, 4, 8)) if gate else 1
            c = _norm("", _log(rng, 1, 16384), groups * 8 * _log(rng, 8, 1024 // groups),
                      rng.choice(("bf16", "fp8", "int8")), groups, gate)
            if c["rows"] * c["dim"] > MOST_NORM:
                continue
        else:
            dim = rng.choice((64, 128))
            kv_heads = rng.choice((1, 2, 4, 8))
            kind = rng.choice(("bf16", "fp8", "int8", "none"))
            b = _draw_batch(rng, 4096)
            kv = b["new_max"] + _log(rng, 1, 1000000 if kind == "none" else 32768)
            c = _rope("", b, (max(b["new_max"], kv // rng.choice((1, 5))), kv), kind,
                      kv_heads * rng.choice((1, 2, 4, 5, 8)), kv_heads, dim,
                      rng.choice((dim, dim, dim // 2, dim // 4)), rng.choice((16, 32, 64, 128)),
                      rng.choice(("half", "half", "neighbours")),
                      rng.choice(("none", "linear", "ramp")))
            if (sum(_lengths(c)) * (c["heads"] + 2 * kv_heads) * dim > MOST_ROPE
                    or (kind != "none" and c["batch"] * kv * kv_heads * dim > MOST_CACHE)):
                continue
        del c["name"]
        return c


def _lengths(case):
    """New tokens of every sequence, from the case alone."""
    rng = random.Random("%d %d %d" % (case["lens"], case["batch"], case["new_max"]))
    out = [1 if b < case["single"] else rng.randint(case["new_min"], case["new_max"])
           for b in range(case["batch"])]
    rng.shuffle(out)   # (the sequences with one token are not the first ones of the batch)
    return out


def _contexts(case):
    """Tokens of every sequence with the new ones counted."""
    rng = random.Random("%d %d" % (case["lens"] + 1, case["kv_max"]))
    return [max(n, rng.randint(case["kv_min"], case["kv_max"])) for n in _lengths(case)]


def work(case):
    op = case["op"]
    if op == "norm":
        n, size = case["rows"] * case["dim"], 2 if case["type"] == "bf16" else 1
        scales = 0 if size == 2 else 4 * case["rows"] * case["groups"]
        # x and gate in; or x and residual in, residual out
        return {"bytes": n * (size + (4 if case["gate"] else 6)) + 4 * case["dim"] + scales,
                "flops": n * (8 if case["gate"] else 5)}
    lens = _lengths(case)
    total, batch = sum(lens), case["batch"]
    if op == "conv":
        c, w = case["channels"], case["width"]
        state = batch * (w - 1) * c * 2
        return {"bytes": 4 * total * c + 2 * state + 4 * c * (w + 1) + 9 * batch,
                "flops": total * c * (2 * w + (4 if case["silu"] else 0))}
    if op == "scan":
        c, n = case["channels"], case["states"]
        state = batch * c * n * (4 if case["pool"] == "fp32" else 2)
        return {"bytes": total * (c * 2 * (4 if case["gate"] else 3) + 4 * n) + 2 * state + 4 * c * (n + 2),
                "flops": total * c * (n * 7 + 12)}
    h, kh, d = case["heads"], case["kv_heads"], case["dim"]
    q, k = total * h * d * 2, total * kh * d * 2
    flops = total * (h + kh) * case["part"] * 3
    if case["type"] == "none":
        return {"bytes": 2 * q + 2 * k + 8 * batch, "flops": flops}
    size = 2 if case["type"] == "bf16" else 1
    row = 2 * total * kh * (d * size + (0 if size == 2 else 4))
    back = 0 if size == 2 else row + 2 * k     # 8-bit rows are read back
    tables = 8 * batch + 4 * sum(-(-kv // case["page"]) for kv in _contexts(case))
    return {"bytes": 2 * q + 2 * k + row + back + tables, "flops": flops + 4 * total * kh * d}


# ------------------------------------------------------------------ the inputs

def frequencies(case):
    """Angles per position of the rotated pairs (64 bits) and the factor m, as a model's
    configuration gives them: base 10000, stretched to four times the context."""
    half = case["part"] // 2
    inv = [10000.0 ** (-i / half) for i in range(half)]
    if case["scaling"] == "linear":
        return [f / 4.0 for f in inv], 1.0
    if case["scaling"] == "ramp":
        # frequencies of fewer than 1 turn in the original 8192 positions are divided by 4,
        # those of more than 32 stay, a ramp lies between
        def dim_of(turns):
            return half * math.log(8192 / (turns * 2 * math.pi)) / math.log(10000.0)
        low, high = max(math.floor(dim_of(32)), 0), min(math.ceil(dim_of(1)), half - 1)
        keep = [1 - min(max((i - low) / max(high - low, 0.001), 0.0), 1.0) for i in range(half)]
        return [f / 4.0 * (1 - k) + f * k for f, k in zip(inv, keep)], 0.1 * math.log(4.0) + 1.0
    return inv, 1.0


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rng = random.Random(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=g, device=dev) * (hi - lo) + lo

    def empty(*shape, like=torch.bfloat16):
        return torch.empty(shape, dtype=like, device=dev)

    s = {"case": case, "op": case["op"]}
    if own:   # the word that a serving loop collects device-side errors in
        import mamba_ssd_chunked_varlen_gb300 as pkg
        s["errors"] = torch.zeros(1, dtype=torch.int32, device=dev)
    if case["op"] == "norm":
        rows, dim = case["rows"], case["dim"]
        # a few columns are larger than the others, and rows differ in size
        column = torch.exp(0.5 * normal(dim))
        s["x"] = (normal(rows, dim) * torch.exp(0.3 * normal(rows, 1))).to(torch.bfloat16)
        s["weight"] = 1 + 0.2 * normal(dim)
        s["gate"] = normal(rows, dim).to(torch.bfloat16) if case["gate"] else None
        s["residual"] = None if case["gate"] else (normal(rows, dim) * column).to(torch.bfloat16)
        if own:
            s["y"] = empty(rows, dim, like=TYPES[case["type"]])
            s["scale"] = None
            if case["type"] != "bf16":
                s["scale"], s["values"] = empty(rows, case["groups"], like=torch.float32), empty(rows, dim)
        return s

    lens = _lengths(case)
    batch, total = case["batch"], sum(lens)
    start = torch.zeros(batch + 1, dtype=torch.int32)
    start[1:] = torch.tensor(lens).cumsum(0)
    s["query_start_loc"], s["total"], s["longest"] = start.to(dev), total, max(lens)
    if case["op"] in ("conv", "scan"):
        c, slots = case["channels"], batch + 3
        order = list(range(slots))
        rng.shuffle(order)
        s["cache_indices"] = torch.tensor(order[:batch], dtype=torch.int32, device=dev)
        # running sequences go on from their slots, some prompts are new
        s["has_initial_state"] = torch.tensor([n == 1 or rng.random() < 0.5 for n in lens], device=dev)
    if case["op"] == "conv":
        w = case["width"]
        s["x"] = normal(total, c).to(torch.bfloat16)
        s["weight"] = normal(c, w) / w ** 0.5
        s["bias"] = 0.2 * normal(c) if case["bias"] else None
        s["conv_pool"] = normal(slots, w - 1, c).to(torch.bfloat16)
        if own:
            s["y"] = empty(total, c)
        return s
    if case["op"] == "scan":
        n = case["states"]
        s["x"] = normal(total, c).to(torch.bfloat16)
        s["dt"] = (0.5 * normal(total, c)).to(torch.bfloat16)
        s["B"], s["C"] = normal(total, n).to(torch.bfloat16), normal(total, n).to(torch.bfloat16)
        s["z"] = normal(total, c).to(torch.bfloat16) if case["gate"] else None
        # decays of one to `states` per unit of the step, steps of 0.001 to 0.1
        s["A"] = -torch.arange(1, n + 1, device=dev) * torch.exp(0.1 * normal(c, n))
        s["D"] = normal(c)
        s["dt_bias"] = torch.log(torch.expm1(torch.exp(uniform(math.log(1e-3), math.log(1e-1), c))))
        s["ssm_pool"] = (0.3 * normal(slots, c, n)).to(TYPES[case["pool"]])
        if own:
            s["y"] = empty(total, c)
            s["workspace"] = pkg.alloc_selective_scan_workspace(total, batch, c, n)
        return s

    h, kh, d, page = (case[k] for k in ("heads", "kv_heads", "dim", "page"))
    contexts = _contexts(case)
    s["kv_lens"] = torch.tensor(contexts, dtype=torch.int32, device=dev)
    s["q"] = normal(total, h, d).to(torch.bfloat16)
    s["k"] = (normal(total, kh, d) * torch.exp(0.3 * normal(total, kh, 1))).to(torch.bfloat16)
    freqs, s["magnitude"] = frequencies(case)
    s["frequencies"] = torch.tensor(freqs, dtype=torch.float64, device=dev)
    if case["type"] != "none":
        s["v"] = normal(total, kh, d).to(torch.bfloat16)
        need = [-(-kv // page) for kv in contexts]
        pages = sum(need) + 3
        order = list(range(pages))
        rng.shuffle(order)
        table = torch.zeros((batch, max(need)), dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        s["block_table"] = table.to(dev)
        s["k_scale"] = s["v_scale"] = None
        for name in ("k", "v"):
            s[name + "_cache"] = torch.zeros((pages, kh, page, d), device=dev).to(TYPES[case["type"]])
            if case["type"] != "bf16":
                s[name + "_scale"] = torch.zeros((pages, kh, page), device=dev)
    if own:
        s["table"] = pkg.alloc_rope_table(freqs)
        s["q_out"], s["k_out"], s["v_out"] = empty(total, h, d), empty(total, kh, d), empty(total, kh, d)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    if not own:
        return {"conv": _plain_conv, "scan": _plain_scan, "norm": _plain_norm, "rope": _plain_rope}[s["op"]](s)
    import mamba_ssd_chunked_varlen_gb300 as pkg
    case = s["case"]
    if s["op"] == "norm":
        pkg.ssd_rms_norm_fwd(s["y"], s["x"], s["weight"], residual=s["residual"], gate=s["gate"],
                             scale=s["scale"], ngroups=case["groups"], eps=EPS)
        if case["type"] == "bf16":
            return {"y": s["y"], "residual": s["residual"]}
        # (torch does not multiply fp8)
        y = s["y"].to(torch.bfloat16) if case["type"] == "fp8" else s["y"]
        torch.mul(y.unflatten(1, (case["groups"], -1)), s["scale"][..., None],
                  out=s["values"].unflatten(1, (case["groups"], -1)))
        return {"y": s["values"], "scale": s["scale"], "residual": s["residual"]}
    if s["op"] == "conv":
        pkg.ssd_causal_conv_varlen_fwd(s["y"], s["x"], s["weight"], s["bias"], s["conv_pool"],
                                       s["query_start_loc"], s["has_initial_state"], s["cache_indices"],
                                       silu=case["silu"], errors=s["errors"])
        return {"y": s["y"], "conv_pool": s["conv_pool"]}
    if s["op"] == "scan":
        pkg.ssd_selective_scan_varlen_fwd(s["y"], s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"],
                                          s["dt_bias"], s["ssm_pool"], s["query_start_loc"],
                                          s["has_initial_state"], s["cache_indices"],
                                          workspace=s["workspace"], errors=s["errors"])
        return {"y": s["y"], "ssm_pool": s["ssm_pool"]}
    how = dict(interleaved=case["pairs"] == "neighbours", magnitude=s["magnitude"], errors=s["errors"])
    if case["type"] == "none":
        pkg.ssd_rope_varlen_fwd(s["q_out"], s["q"], s["k_out"], s["k"], s["table"], s["query_start_loc"],
                                s["kv_lens"], **how)
        return {"q": s["q_out"], "k": s["k_out"]}
    cache = (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    where = (s["query_start_loc"], s["kv_lens"], s["block_table"])
    pkg.ssd_rope_kv_cache_write(s["q_out"], s["q"], s["k"], s["v"], s["table"], *cache, *where, **how)
    if case["type"] == "bf16":
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    pkg.ssd_kv_cache_read(s["k_out"], s["v_out"], *cache, *where, errors=s["errors"])
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


# ------------------------------------------------------------------ the plain forms

def _codes(x, kind):
    """Codes and scales of rows (the last axis), 32 bits until the code."""
    a = x.abs().amax(-1).clamp(min=TINY)
    top = torch.full_like(a, TOP[kind])   # (a quotient with a number would go by its reciprocal)
    y = x * (top / a).unsqueeze(-1)
    code = y.round().to(torch.int8) if kind == "int8" else y.to(torch.float8_e4m3fn)
    return code, a / top


def _silu(x):
    return x / (1 + torch.exp(-x))


def _plain_norm(s):
    case = s["case"]
    x = s["x"].float()
    if case["gate"]:
        x = x * _silu(s["gate"].float())
    else:
        x = x + s["residual"].float()
        s["residual"].copy_(x)
    x = x.unflatten(1, (case["groups"], -1))
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["weight"].view(case["groups"], -1)
    if case["type"] == "bf16":
        return {"y": y.flatten(1).to(torch.bfloat16), "residual": s["residual"]}
    code, scale = _codes(y, case["type"])
    values = (code.float() * scale[..., None]).to(torch.bfloat16).flatten(1)
    return {"y": values, "scale": scale, "residual": s["residual"]}


def _places(s):
    """Sequence of every token and its place in it."""
    start = s["query_start_loc"].long()
    t = torch.arange(s["total"], device=start.device)
    b = torch.searchsorted(start, t, right=True) - 1
    return b, t - start[b]


def _first_states(s, pool):
    keep = s["has_initial_state"].view(-1, 1, 1)
    return torch.where(keep, s[pool][s["cache_indices"].long()].float(), 0.0)


def _plain_conv(s):
    case, start = s["case"], s["query_start_loc"].long()
    w = case["width"]
    x, first = s["x"].float(), _first_states(s, "conv_pool")
    b, p = _places(s)
    j = torch.arange(w, device=x.device)
    at = p[:, None] + j - (w - 1)                      # the taps' places, before the start: the state's
    t = torch.arange(s["total"], device=x.device)[:, None] + j - (w - 1)
    taps = torch.where((at >= 0)[..., None], x[t.clamp(min=0)], first[b[:, None], (at + w - 1).clamp(max=w - 2)])
    y = (taps * s["weight"].t()).sum(1)
    if case["bias"]:
        y = y + s["bias"]
    if case["silu"]:
        y = _silu(y)
    n = (start[1:] - start[:-1])[:, None]
    at = n + j[:-1] - (w - 1)                          # the last inputs of every sequence
    last = torch.where((at >= 0)[..., None], x[(start[:-1, None] + at).clamp(min=0, max=s["total"] - 1)],
                       torch.gather(first, 1, (at + w - 1).clamp(max=w - 2)[..., None].expand_as(first)))
    s["conv_pool"][s["cache_indices"].long()] = last.to(torch.bfloat16)
    return {"y": y.to(torch.bfloat16), "conv_pool": s["conv_pool"]}


def _plain_scan(s):
    start, slots = s["query_start_loc"].long(), s["cache_indices"].long()
    x, first = s["x"].float(), _first_states(s, "ssm_pool")
    v = s["dt"].float() + s["dt_bias"]
    d = torch.where(v > 20, v, torch.log1p(torch.exp(v)))
    a = torch.exp(d[..., None] * s["A"])
    h = (d * x)[..., None] * s["B"].float()[:, None]
    # a sequence's first token takes its state in, and nothing of the token before it
    begin, n = start[:-1], start[1:] - start[:-1]
    some = n > 0
    h[begin[some]] += a[begin[some]] * first[some]
    a[begin[some]] = 0
    step = 1
    while step < s["longest"]:
        new = h.clone()
        new[step:].addcmul_(a[step:], h[:-step])
        h = new
        a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    del a
    y = (h * s["C"].float()[:, None]).sum(-1) + s["D"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    s["ssm_pool"][slots] = torch.where(some.view(-1, 1, 1), h[(start[1:] - 1).clamp(min=0)], first).to(s["ssm_pool"].dtype)
    return {"y": y.to(torch.bfloat16), "ssm_pool": s["ssm_pool"]}


def _rotate(s, x, cos, sin):
    part, half = s["case"]["part"], s["case"]["part"] // 2
    x = x.float()
    r, rest = x[..., :part], x[..., part:]
    if s["case"]["pairs"] == "half":
        a, b = r[..., :half], r[..., half:]
    else:
        a, b = r[..., 0::2], r[..., 1::2]
    out = (a * cos - b * sin, b * cos + a * sin)
    r = torch.cat(out, -1) if s["case"]["pairs"] == "half" else torch.stack(out, -1).flatten(-2)
    return torch.cat((r, rest), -1)


def _plain_rope(s):
    case, start = s["case"], s["query_start_loc"].long()
    b, p = _places(s)
    at = s["kv_lens"].long()[b] - (start[b + 1] - start[b]) + p
    angle = at.double()[:, None] * s["frequencies"]
    cos, sin = ((f(angle) * s["magnitude"]).float()[:, None] for f in (torch.cos, torch.sin))
    q, k = _rotate(s, s["q"], cos, sin), _rotate(s, s["k"], cos, sin)
    out = {"q": q.to(torch.bfloat16)}
    if case["type"] == "none":
        return out | {"k": k.to(torch.bfloat16)}
    page, row = s["block_table"].long()[b, at // case["page"]], at % case["page"]
    for name, x in (("k", k), ("v", s["v"].float())):
        if case["type"] == "bf16":
            s[name + "_cache"][page, :, row] = x.to(torch.bfloat16)
            out[name + "_cache"] = s[name + "_cache"]
            continue
        code, scale = _codes(x, case["type"])
        # (torch has no indexed store of fp8: its bytes are stored)
        s[name + "_cache"].view(torch.int8)[page, :, row] = code.view(torch.int8)
        s[name + "_scale"][page, :, row] = scale
        back = s[name + "_cache"].view(torch.int8)[page, :, row].view(code.dtype).float()
        out[name] = (back * s[name + "_scale"][page, :, row][..., None]).to(torch.bfloat16)
        out[name + "_scale"] = s[name + "_scale"]
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


def _exact_norm(case, s):
    x = s["x"].double()
    if case["gate"]:
        z = s["gate"].double()
        x = x * z * torch.sigmoid(z)
        kept = None
    else:
        x = kept = x + s["residual"].double()
    groups = x.chunk(case["groups"], 1)
    y = [v / torch.sqrt(v.square().mean(1, keepdim=True) + EPS) for v in groups]
    y = [v * w for v, w in zip(y, s["weight"].double().chunk(case["groups"]))]
    if case["type"] == "bf16":
        return {"y": torch.cat(y, 1), "residual": kept}
    coded = [_exact_codes(v, case["type"]) for v in y]
    return {"y": torch.cat([c * a[:, None] for c, a in coded], 1), "scale": torch.stack([a for _, a in coded], 1),
            "residual": kept}


def _exact_conv(case, s, lens):
    w, at, y, pool = case["width"], 0, [], s["conv_pool"].double()
    for b, n in enumerate(lens):
        slot = int(s["cache_indices"][b])
        before = pool[slot] if s["has_initial_state"][b] else torch.zeros_like(pool[slot])
        line = torch.cat((before, s["x"][at:at + n].double()))
        out = sum(line[j:j + n] * s["weight"][:, j].double() for j in range(w))
        if case["bias"]:
            out = out + s["bias"].double()
        y.append(out * torch.sigmoid(out) if case["silu"] else out)
        pool[slot] = line[n:]
        at += n
    return {"y": torch.cat(y), "conv_pool": pool}


def _exact_scan(case, s, lens):
    if max(lens) * max(1.0, case["batch"] * case["channels"] * case["states"] / 1e6) > 2e5:
        return None   # over about 20 s, token by token
    pool = s["ssm_pool"].double()
    x, A = s["x"].double(), s["A"].double()
    d = torch.nn.functional.softplus(s["dt"].double() + s["dt_bias"].double(), threshold=50)
    B, C = s["B"].double(), s["C"].double()
    y = torch.empty_like(x)
    # the sequences by falling length: at step i the first ones are still running
    order = sorted(range(len(lens)), key=lambda b: -lens[b])
    slots = s["cache_indices"].long()[order]
    h = torch.where(s["has_initial_state"][order].view(-1, 1, 1), pool[slots], 0.0)
    start = s["query_start_loc"].long()[:-1][order]
    running = len(order)
    for i in range(max(lens)):
        while lens[order[running - 1]] <= i:
            running -= 1
        t = start[:running] + i
        h[:running] *= torch.exp(d[t][..., None] * A)
        h[:running] += (d[t] * x[t])[..., None] * B[t][:, None]
        y[t] = torch.einsum("bcn,bn->bc", h[:running], C[t])
    pool[slots] = h
    y += s["D"].double() * x
    if s["z"] is not None:
        y *= s["z"].double() * torch.sigmoid(s["z"].double())
    return {"y": y, "ssm_pool": pool}


def _exact_rope(case, s, lens):
    freqs, m = frequencies(case)
    contexts = _contexts(case)
    at = torch.cat([torch.arange(kv - n, kv, dtype=torch.float64) for n, kv in zip(lens, contexts)]).cuda()
    turn = torch.polar(torch.full((at.numel(), len(freqs)), m, dtype=torch.float64, device="cuda"),
                       torch.outer(at, torch.tensor(freqs, dtype=torch.float64, device="cuda")))[:, None]
    part = case["part"]

    def rotated(x):
        r = x[..., :part].double()
        if case["pairs"] == "neighbours":
            r = torch.view_as_real(torch.view_as_complex(r.unflatten(-1, (-1, 2)).contiguous()) * turn).flatten(-2)
        else:
            v = torch.complex(r[..., :part // 2], r[..., part // 2:]) * turn
            r = torch.cat((v.real, v.imag), -1)
        return torch.cat((r, x[..., part:].double()), -1)

    out, k = {"q": rotated(s["q"])}, rotated(s["k"])
    if case["type"] == "none":
        return out | {"k": k}
    for name, x in (("k", k), ("v", s["v"].double())):
        if case["type"] == "bf16":
            rows, scales = x, None
            kept = s[name + "_cache"].double()
        else:
            code, scales = _exact_codes(x, case["type"])
            rows = out[name] = code * scales[..., None]
            kept = s[name + "_scale"].double()
        t = 0
        for b, (n, kv) in enumerate(zip(lens, contexts)):
            j = torch.arange(kv - n, kv, device=x.device)
            page = s["block_table"][b].long()[j // case["page"]]
            kept[page, :, j % case["page"]] = (rows if scales is None else scales)[t:t + n]
            t += n
        out[name + ("_cache" if scales is None else "_scale")] = kept
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(case, s)
    return {"conv": _exact_conv, "scan": _exact_scan, "rope": _exact_rope}[case["op"]](case, s, _lengths(case))
