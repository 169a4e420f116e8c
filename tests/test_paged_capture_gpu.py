"""The paged-cache operators captured as a process's first calls, and replayed on lengths, tables and queries other than those that
were captured."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from test_kv8_attn_gpu import Case
from top_sparse_mla_gb300 import native

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from top_sparse_mla_gb300.build import build
    build()
    native.library()


def _captured(call):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    return graph


def first_calls(which):
    """One operator's first call of the process is captured (no warm-up), replayed and checked."""
    if which == "map":
        i32 = dict(dtype=torch.int32, device="cuda")
        ctx, new, table, free = (torch.tensor(x, **i32) for x in ([3, 0], [2, 5], [[9, -1], [-1, -1]], [20, 21, 22]))
        cu, kv, pos, info = (torch.zeros(n, **i32) for n in (3, 2, 8, 2))
        slots = torch.zeros(8, dtype=torch.int64, device="cuda")
        _captured(lambda: native.dsa_page_map(ctx, new, table, free, 4, cu, kv, pos, slots, None, info)).replay()
        assert slots.tolist() == [39, 80, 84, 85, 86, 87, 88, -1] and info.tolist() == [3, 0]
    elif which == "insert":
        k = torch.full((3, 1, 64), 2.0, dtype=torch.bfloat16, device="cuda")
        pools = [torch.zeros((2, 1, 16, 64), dtype=torch.uint8, device="cuda") for _ in range(2)]
        scales = [torch.ones((2, 1), device="cuda") for _ in range(2)]
        slots = torch.tensor([16, 17, 18], device="cuda")
        _captured(lambda: native.dsa_kv8_insert(k, k, slots, *pools, *scales)).replay()
        assert (pools[0][1, 0, :3] == 0x78).all() and scales[1][1, 0].item() == 2.0 ** -7   # 2 = 256 * 2^-7
    else:
        lens = {"rows": [(1, 700), (2, 90)], "many rows": [(1, 20)] * 3000, "tiles": [(40, 300)] * 90, "cluster": [(33, 2100)]}[which]
        c = Case(97, lens, h=1, g=8, d=64, page=32)
        D = c.device()
        p = native.dsa_kv8_params_init(D["q"], D["kp"], D["table"], max_q_len=max(q for q, _ in lens))
        p.softmax_scale = c.scale
        out = torch.full((c.n, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((c.n, 8), 7.0, device="cuda")
        ws = torch.empty(native.dsa_kv8_attn_workspace_size(p), dtype=torch.uint8, device="cuda")
        _captured(lambda: native.dsa_kv8_attn_fwd(D["q"], D["kp"], D["vp"], D["ks"], D["vs"], D["table"], D["cu"], D["kv"], out, p, ws,
                                                  lse=lse)).replay()
        torch.cuda.synchronize()
        c.check(out, lse)


@pytest.mark.parametrize("which", ["map", "insert", "rows", "many rows", "tiles", "cluster"])
def test_a_process_s_first_call_may_be_captured(which):
    code = f"import test_paged_capture_gpu as t; t.first_calls({which!r})"
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([here, os.path.dirname(here), os.environ.get("PYTHONPATH", "")]))
    run = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]


@pytest.mark.parametrize("most,group,window", [(1, 8, 0), (4, 8, 0), (40, 4, 0), (40, 16, 77), (200, 2, 0)])
def test_replayed_on_other_lengths_tables_and_queries(most, group, window):
    """A step of 12 requests with room for 64 pages each, captured once and replayed on batches of other lengths."""
    rng = np.random.default_rng(most + group)
    n, cols, page, rows = 12, 64, 16, 12 * most + 3

    def batch(seed):
        lens = [(int(q), int(rng.integers(q, cols * page + 1))) for q in rng.integers(0, most + 1, n)]
        c = Case(seed, lens, h=2, g=group, d=64, page=page, window=window)
        table = np.full((n, cols), -1, np.int32)
        table[:, :c.table.shape[1]] = c.table[:, :cols]
        c.table = table
        pad = rows - c.n
        c.q = torch.cat([c.q, torch.full((pad,) + c.q.shape[1:], float("nan"), dtype=c.q.dtype)])
        c.n = rows
        pools = n * cols + 3   # as many pages for every batch
        for name in ("kp", "vp", "ks", "vs"):
            x = getattr(c, name)
            setattr(c, name, np.concatenate([x, np.zeros((pools - x.shape[0],) + x.shape[1:], x.dtype)]))
        c.table[c.table >= x.shape[0]] = -1   # entries that named no page must not name one of the new
        return c

    first = batch(0)
    D = first.device()
    p = native.dsa_kv8_params_init(D["q"], D["kp"], D["table"], max_q_len=most, window=window, softmax_scale=first.scale)
    out = torch.empty((rows, 2 * group, 64), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((rows, 2 * group), device="cuda")
    ws = torch.empty(native.dsa_kv8_attn_workspace_size(p), dtype=torch.uint8, device="cuda")
    graph = _captured(lambda: native.dsa_kv8_attn_fwd(D["q"], D["kp"], D["vp"], D["ks"], D["vs"], D["table"], D["cu"], D["kv"], out, p,
                                                      ws, lse=lse))
    for seed in range(4):
        c = first if seed == 0 else batch(seed)
        for name, x in c.device().items():
            D[name].copy_(x)
        out.fill_(7.0)
        lse.fill_(7.0)
        graph.replay()
        assert native.dsa_sparse_attn_read_status(ws) == 0
        c.check(out, lse)
