"""One block of a hybrid model served with continuous batching: a Mamba-2 scan
layer and an attention layer on the same ragged batch.

Every step takes the new tokens of all running sequences, prompts and single
tokens alike, as one batch described by ``query_start_loc``:

    scan layer       ssd_scan_varlen_fwd_strided  on column views of a projection,
                     recurrent states in a pool of slots
    attention layer  ssd_kv_cache_write  k and v of the new tokens into pages
                     ssd_attn_varlen_fwd  the new tokens over the whole context

    python examples/hybrid_serving.py [--cache bfloat16|float8_e4m3fn|int8]

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
                 device="cuda"):
        g = torch.Generator().manual_seed(seed)

        def weight(n, m):
            return (torch.randn(n, m, generator=g) / n ** 0.5).bfloat16().to(device)

        inner, gn = SCAN["nheads"] * SCAN["head_dim"], SCAN["ngroups"] * SCAN["dstate"]
        self.scan_cols = [inner, gn, gn, SCAN["nheads"]]             # x, B, C, dt
        self.attn_cols = [HEADS * DIM, KV_HEADS * DIM, KV_HEADS * DIM]
        self.scan_in, self.scan_out = weight(HIDDEN, sum(self.scan_cols)), weight(inner, HIDDEN)
        self.attn_in, self.attn_out = weight(HIDDEN, sum(self.attn_cols)), weight(HEADS * DIM, HIDDEN)
        n = SCAN["nheads"]
        self.A = -torch.rand(n, generator=g).add(0.5).to(device)
        self.D = torch.ones(n, device=device)
        self.dt_bias = torch.full((n,), -2.0, device=device)
        # what a server keeps: the states, the pages, the workspaces, one word of errors
        self.states = torch.zeros(slots, n, SCAN["head_dim"], SCAN["dstate"], device=device)
        width = (max_context + PAGE - 1) // PAGE
        self.pages = Pages(slots * width, slots, width)
        shape = (slots * width, KV_HEADS, PAGE, DIM)
        self.k_cache = torch.zeros(shape, device=device).to(cache)
        self.v_cache = self.k_cache.clone()
        quantised = cache is not torch.bfloat16
        self.k_scale = torch.zeros(shape[:3], device=device) if quantised else None
        self.v_scale = self.k_scale.clone() if quantised else None
        self.errors = torch.zeros(1, dtype=torch.int32, device=device)
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

        # ---- the scan layer: column views of one projection
        x, B, C, dt = (h @ self.scan_in).split(self.scan_cols, 1)
        y = torch.empty(total, SCAN["nheads"], SCAN["head_dim"], dtype=torch.bfloat16, device=device)
        ssd.ssd_scan_varlen_fwd_strided(
            y, x.unflatten(1, (SCAN["nheads"], -1)), dt, self.A, B.unflatten(1, (SCAN["ngroups"], -1)),
            C.unflatten(1, (SCAN["ngroups"], -1)), self.D, self.dt_bias, self.states, query_start_loc,
            torch.tensor([not f for f in fresh], device=device), torch.tensor(slots, **i32),
            chunk_size=SCAN["chunk_size"], workspace=self.scan_ws)
        h = h + y.flatten(1) @ self.scan_out

        # ---- the attention layer: the new keys and values first, then the queries
        q, k, v = (h @ self.attn_in).split(self.attn_cols, 1)
        q = q.unflatten(1, (HEADS, DIM))
        k, v = (t.unflatten(1, (KV_HEADS, DIM)) for t in (k, v))
        ssd.ssd_kv_cache_write(k, v, *self.cache, *self.batch, errors=self.errors)
        o = torch.empty(total, HEADS, DIM, dtype=torch.bfloat16, device=device)
        ssd.ssd_attn_varlen_fwd(o, None, q, *self.cache, *self.batch, softmax_scale=DIM ** -0.5,
                                workspace=self.attn_ws, errors=self.errors)
        self.last = q, o
        return h + o.flatten(1) @ self.attn_out

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
    p.add_argument("--steps", type=int, default=12)
    a = p.parse_args()
    block = HybridBlock(cache=getattr(torch, a.cache))
    for i, (batch, out) in enumerate(serve(block, a.steps)):
        print(f"step {i}: {sum(n for _, n in batch)} new tokens of {len(batch)} sequences, "
              f"contexts {[block.lens[s] for s, _ in batch]}, rms {out.float().pow(2).mean().sqrt().item():.3f}")
    flags = int(block.errors) | ssd.ssd_scan_varlen_read_errors(block.scan_ws)
    print(f"device error flags: {flags:#x}")
    return 1 if flags else 0


if __name__ == "__main__":
    sys.exit(main())
