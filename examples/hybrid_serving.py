"""One block of a hybrid model served with continuous batching: a scan layer and an
attention layer on the same ragged batch.

Every step takes the new tokens of all running sequences, prompts and single
tokens alike, as one batch described by ``query_start_loc``:

    scan layer       ssd_rms_norm_fwd             the layer's input
                     ssd_causal_conv_varlen_fwd   columns of a projection, the last
                     inputs in a pool of slots
                     ssd_scan_varlen_fwd_strided  on column views of the result,
                     recurrent states in a pool of slots; or, with a step and decays of
                     each channel's own, ssd_selective_scan_varlen_fwd
                     ssd_rms_norm_fwd             the gated output, in groups
    attention layer  ssd_rms_norm_fwd             its input, with the residual's addition
                     ssd_rope_kv_cache_write      q, and k and v into pages, rotated
                     ssd_attn_varlen_fwd          the new tokens over the whole context

    python examples/hybrid_serving.py [--cache bfloat16|float8_e4m3fn|int8] [--scan ssd|selective]

The weights are random and the projections plain matrix products: what is shown
is how the calls share a batch.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mamba_ssd_chunked_varlen_gb300 as ssd  # noqa: E402

HIDDEN = 512
SCAN = dict(nheads=16, head_dim=64, ngroups=1, dstate=128, chunk_size=128)
SELECTIVE = dict(channels=1024, dstate=16, step_rank=32)
CONV, GROUPS = 4, 2     # the convolution's width, groups of the gated norm
HEADS, KV_HEADS, DIM, PAGE = 16, 4, 128, 16


class Pages:
    """Pages of the cache and the block table of the running sequences."""

    def __init__(self, num_pages, slots, width):
        self.free = list(range(num_pages))[::-1]
        self.table = [[] for _ in range(slots)]
        self.width = width

    def reserve(self, slot, tokens):
        while len(self.table[slot]) * PAGE < tokens:
            self.table[slot].append(self.free.pop())

    def rows(self, slots, device):
        t = [self.table[s] + [0] * (self.width - len(self.table[s])) for s in slots]
        return torch.tensor(t, dtype=torch.int32, device=device)


class HybridBlock:
    def __init__(self, slots=8, max_tokens=1024, max_context=1024, cache=torch.bfloat16, seed=0,
                 device="cuda", scan="ssd"):
        g = torch.Generator().manual_seed(seed)

        def weight(n, m):
            return (torch.randn(n, m, generator=g) / n ** 0.5).bfloat16().to(device)

        def near_one(*shape):
            return torch.rand(shape, generator=g).add(0.5).to(device)

        inner, gn = SCAN["nheads"] * SCAN["head_dim"], SCAN["ngroups"] * SCAN["dstate"]
        self.selective = scan == "selective"
        n = SCAN["nheads"]
        if self.selective:
            inner, d, rank = SELECTIVE["channels"], SELECTIVE["dstate"], SELECTIVE["step_rank"]
            self.conv_cols = [inner]
            self.scan_cols = [inner, inner]                          # z, x
            self.step_in, self.step_out = weight(inner, rank + 2 * d), weight(rank, inner)
            self.A, n = -near_one(inner, d) * torch.arange(1, d + 1, device=device), inner
        else:
            self.conv_cols = [inner, gn, gn]                         # x, B, C
            self.scan_cols = [inner, sum(self.conv_cols), n]         # z, the convolution's, dt
            self.A = -near_one(n)
        self.D = torch.ones(n, device=device)
        self.dt_bias = torch.full((n,), -2.0, device=device)
        self.conv_weight, self.conv_bias = near_one(sum(self.conv_cols), CONV) - 0.9, None
        self.norms = near_one(HIDDEN), near_one(inner), near_one(HIDDEN)
        self.attn_cols = [HEADS * DIM, KV_HEADS * DIM, KV_HEADS * DIM]
        self.scan_in, self.scan_out = weight(HIDDEN, sum(self.scan_cols)), weight(inner, HIDDEN)
        self.attn_in, self.attn_out = weight(HIDDEN, sum(self.attn_cols)), weight(HEADS * DIM, HIDDEN)
        frequencies, self.magnitude = ssd.rope_frequencies(DIM)
        self.turns = ssd.alloc_rope_table(frequencies, device)
        # what a server keeps: the states, the pages, the workspaces, one word of errors
        self.conv_states = torch.zeros(slots, CONV - 1, sum(self.conv_cols), dtype=torch.bfloat16, device=device)
        state = (inner, SELECTIVE["dstate"]) if self.selective else (n, SCAN["head_dim"], SCAN["dstate"])
        self.states = torch.zeros(slots, *state, device=device)
        width = (max_context + PAGE - 1) // PAGE
        self.pages = Pages(slots * width, slots, width)
        shape = (slots * width, KV_HEADS, PAGE, DIM)
        self.k_cache = torch.zeros(shape, device=device).to(cache)
        self.v_cache = self.k_cache.clone()
        quantised = cache is not torch.bfloat16
        self.k_scale = torch.zeros(shape[:3], device=device) if quantised else None
        self.v_scale = self.k_scale.clone() if quantised else None
        self.errors = torch.zeros(1, dtype=torch.int32, device=device)
        if self.selective:
            self.scan_ws = ssd.alloc_selective_scan_workspace(max_tokens, slots, *state, device=device)
        else:
            self.scan_ws = ssd.alloc_workspace(max_tokens, slots, n, SCAN["head_dim"], SCAN["ngroups"],
                                               SCAN["dstate"], SCAN["chunk_size"], device=device)
        self.attn_ws = ssd.alloc_attn_workspace(max_tokens, slots, HEADS, KV_HEADS, DIM, device=device)
        self.lens = [0] * slots
        self.device = device

    @property
    def cache(self):
        return self.k_cache, self.v_cache, self.k_scale, self.v_scale

    def step(self, h, batch):
        """h (tokens, hidden) bf16: the new tokens of the sequences in `batch`, a list
        of (slot, number of new tokens); each new sequence starts in a slot whose
        length is 0."""
        device, total = self.device, h.shape[0]
        slots = [s for s, _ in batch]
        starts = [0]
        for s, n in batch:
            starts.append(starts[-1] + n)
            self.pages.reserve(s, self.lens[s] + n)
        fresh = [self.lens[s] == 0 for s in slots]
        for s, n in batch:
            self.lens[s] += n
        i32 = dict(dtype=torch.int32, device=device)
        query_start_loc = torch.tensor(starts, **i32)
        kv_lens = torch.tensor([self.lens[s] for s in slots], **i32)
        block_table = self.pages.rows(slots, device)
        self.batch = query_start_loc, kv_lens, block_table
        where = (query_start_loc, torch.tensor([not f for f in fresh], device=device),
                 torch.tensor(slots, **i32))

        # ---- the scan layer: column views of one projection, the gate first
        residual, normed = h.clone(), torch.empty_like(h)
        ssd.ssd_rms_norm_fwd(normed, h, self.norms[0])
        z, x, *dt = (normed @ self.scan_in).split(self.scan_cols, 1)
        mixed = torch.empty(total, sum(self.conv_cols), dtype=torch.bfloat16, device=device)
        ssd.ssd_causal_conv_varlen_fwd(mixed, x, self.conv_weight, self.conv_bias, self.conv_states, *where,
                                       errors=self.errors)
        y = torch.empty(total, z.shape[1], dtype=torch.bfloat16, device=device)
        if self.selective:
            self.scan_selective(y, mixed, where)
        else:
            self.scan_heads(y, mixed, dt[0], where)
        ssd.ssd_rms_norm_fwd(y, y, self.norms[1], gate=z, ngroups=GROUPS)

        # ---- the attention layer: the new keys and values with the queries' rotation first
        ssd.ssd_rms_norm_fwd(normed, y @ self.scan_out, self.norms[2], residual=residual)
        q, k, v = (normed @ self.attn_in).split(self.attn_cols, 1)
        k, v = (t.unflatten(1, (KV_HEADS, DIM)) for t in (k, v))
        plain, q = q.unflatten(1, (HEADS, DIM)), torch.empty(total, HEADS, DIM, dtype=torch.bfloat16, device=device)
        ssd.ssd_rope_kv_cache_write(q, plain, k, v, self.turns, *self.cache, *self.batch,
                                    magnitude=self.magnitude, errors=self.errors)
        o = torch.empty(total, HEADS, DIM, dtype=torch.bfloat16, device=device)
        ssd.ssd_attn_varlen_fwd(o, None, q, *self.cache, *self.batch, softmax_scale=DIM ** -0.5,
                                workspace=self.attn_ws, errors=self.errors)
        self.last = q, o
        return residual + o.flatten(1) @ self.attn_out

    def scan_heads(self, y, mixed, dt, where):
        """The scan whose step and decay are each head's."""
        x, B, C = mixed.split(self.conv_cols, 1)
        ssd.ssd_scan_varlen_fwd_strided(
            y.unflatten(1, (SCAN["nheads"], -1)), x.unflatten(1, (SCAN["nheads"], -1)), dt, self.A,
            B.unflatten(1, (SCAN["ngroups"], -1)), C.unflatten(1, (SCAN["ngroups"], -1)), self.D, self.dt_bias,
            self.states, *where, chunk_size=SCAN["chunk_size"], workspace=self.scan_ws)

    def scan_selective(self, y, x, where):
        """The scan whose step and decays are each channel's, made from x."""
        rank, d = SELECTIVE["step_rank"], SELECTIVE["dstate"]
        step, B, C = (x @ self.step_in).split([rank, d, d], 1)
        ssd.ssd_selective_scan_varlen_fwd(y, x, step @ self.step_out, self.A, B, C, self.D, None, self.dt_bias,
                                          self.states, *where, workspace=self.scan_ws, errors=self.errors)

    def flags(self):
        """The device-side errors of all calls so far."""
        return int(self.errors) | (0 if self.selective else ssd.ssd_scan_varlen_read_errors(self.scan_ws))

    def contexts(self):
        """The last step's contexts as the cache has them: k, v (tokens, kv heads, dim)
        bf16 and the sequences' first tokens."""
        _, kv_lens, block_table = self.batch
        first = torch.nn.functional.pad(kv_lens.cumsum(0), (1, 0)).to(torch.int32)
        k = torch.empty(int(first[-1]), KV_HEADS, DIM, dtype=torch.bfloat16, device=self.device)
        v = torch.empty_like(k)
        ssd.ssd_kv_cache_read(k, v, *self.cache, first, kv_lens, block_table, errors=self.errors)
        return k, v, first


def serve(block, steps=12, seed=1):
    """Three prompts, then single tokens; a fourth prompt joins on the way, so that one
    step mixes a prompt with single tokens.  Yields (batch, output) of every step."""
    g = torch.Generator().manual_seed(seed)
    plan = [[(0, 300), (1, 17), (2, 1)]] + [[(0, 1), (1, 1), (2, 1)]] * 3
    plan += [[(0, 1), (1, 1), (2, 1), (3, 129)]] + [[(s, 1) for s in range(4)]] * max(steps - 5, 0)
    for batch in plan[:steps]:
        tokens = sum(n for _, n in batch)
        h = torch.randn(tokens, HIDDEN, generator=g).bfloat16().to(block.device)
        yield batch, block.step(h, batch)


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--cache", default="bfloat16", choices=("bfloat16", "float8_e4m3fn", "int8"))
    p.add_argument("--scan", default="ssd", choices=("ssd", "selective"))
    p.add_argument("--steps", type=int, default=12)
    a = p.parse_args()
    block = HybridBlock(cache=getattr(torch, a.cache), scan=a.scan)
    for i, (batch, out) in enumerate(serve(block, a.steps)):
        print(f"step {i}: {sum(n for _, n in batch)} new tokens of {len(batch)} sequences, "
              f"contexts {[block.lens[s] for s, _ in batch]}, rms {out.float().pow(2).mean().sqrt().item():.3f}")
    flags = block.flags()
    print(f"device error flags: {flags:#x}")
    return 1 if flags else 0


if __name__ == "__main__":
    sys.exit(main())
