"""Calls of different batches in turn, in one workspace and without a stop between: each call's
kernels go by its own block table and lists, also where they start ahead of their
predecessor's end."""
from __future__ import annotations

import numpy as np
import pytest

from mamba_ssd_chunked_varlen_gb300 import workloads as W

from helpers import run_cuda, to_device

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def test_calls_in_a_row_have_tables_of_their_own():
    import mamba_ssd_chunked_varlen_gb300 as pkg
    rng = np.random.default_rng(5)
    made, most = [], 0
    for n, lengths in enumerate(([300, 129, 5, 2049], [1024, 12, 64], [13, 256, 777, 128, 1])):
        lens = []
        while sum(lens) < 60_000:
            lens.append(int(rng.choice(lengths)))
        w = W.make_workload(f"row{n}", lens, 8, 64, 2, 128, 128, max_slots=len(lens) + 3, seed=60 + n,
                            has_init_p=0.5)
        # (with the block table)
        assert pkg.ssd_scan_varlen_num_launches(w.total_len, w.batch, w.nheads, w.head_dim, w.ngroups,
                                                w.dstate, w.chunk_size) == 5
        y, pool, _, _ = run_cuda(w)
        made.append((w, to_device(w), y, pool.clone()))
        most = max(most, pkg.ssd_scan_varlen_workspace_size(w.total_len, w.batch, w.nheads, w.head_dim,
                                                            w.ngroups, w.dstate, w.chunk_size))
    ws = torch.empty(most, dtype=torch.uint8, device="cuda")
    first = [d["ssm_pool"].clone() for _, d, _, _ in made]
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(10):
        out = []
        for (w, d, _, _), pool in zip(made, first):
            d["ssm_pool"].copy_(pool)
        for w, d, _, _ in made:
            out.append(run_cuda(w, dev=d, workspace=ws)[0])
        for y2, (_, d, y, pool) in zip(out, made):
            wrong += (y2.view(torch.int16) != y.view(torch.int16)).sum()
            wrong += (d["ssm_pool"].view(torch.int32) != pool.view(torch.int32)).sum()
    assert wrong.item() == 0
