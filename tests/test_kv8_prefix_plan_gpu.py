"""Each call of the attention for requests that share prefixes goes by its own plan, whatever a call before left in the workspace and
in the caches.  (The tiles' kernel begins while the one in front of it is on its way, and takes the plan by a word that the plan
kernel releases and the last kernel clears.)"""

import numpy as np
import pytest
import torch

from test_kv8_prefix_gpu import PrefixCase, _lib  # noqa: F401
from top_sparse_mla_gb300 import native

pytestmark = pytest.mark.gpu


def _batches(D, c, seed, n):
    """Lengths and prefixes of n batches of c's shape: requests of other lengths, groups of other sizes."""
    rng = np.random.default_rng(seed)
    out = []
    for _ in range(n):
        kv = np.array([rng.integers(ql, kv + 1) for ql, kv in c.lens], np.int32)
        cut = int(rng.integers(1, len(kv)))
        out.append([torch.from_numpy(np.asarray(x, np.int32)).cuda() for x in (kv, [0, cut, len(kv)], [int(rng.integers(0, 700)), 688])])
    return out


@pytest.mark.parametrize("h,n,q", [(1, 60, 1), (8, 60, 4)], ids=["shared out", "in turn"])
def test_calls_one_after_the_other_in_one_workspace(h, n, q):
    # (1, 60): few tiles, whose blocks are shared out; (8, 60) with 32 rows a request and more: tiles in turn
    c = PrefixCase(61, [(q, 700 + i) for i in range(n)], [(n, 688)], page=16, h=h, g=8 if q == 1 else 16, d=64)
    D = c.device()
    p = native.dsa_kv8_params_init(D["q"], D["kp"], D["table"], max_q_len=q)
    size = native.dsa_kv8_prefix_workspace_size(p, 2)
    batches = _batches(D, c, 62, 6)

    def call(batch, out, lse, ws):
        kv, cug, pre = batch
        native.dsa_kv8_prefix_attn_fwd(D["q"], D["kp"], D["vp"], D["ks"], D["vs"], D["table"], D["cu"], kv, cug, pre, out, p, ws, lse=lse)

    def empty():
        return torch.full_like(D["q"], 7.0), torch.full((c.n, h * c.g), 7.0, device="cuda")

    want = []
    for b in batches:
        out, lse = empty()
        ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
        call(b, out, lse, ws)
        assert native.dsa_sparse_attn_read_status(ws) == 0
        want.append((out, lse))
    assert not torch.equal(want[0][0], want[1][0])

    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    got = [empty() for _ in range(10 * len(batches))]
    for i, (out, lse) in enumerate(got):
        call(batches[i % len(batches)], out, lse, ws)
    assert native.dsa_sparse_attn_read_status(ws) == 0
    for i, pair in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(pair, want[i % len(batches)])), i

    # as a graph, beside calls of its own between its launches
    got = [empty() for _ in batches]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            for b, (out, lse) in zip(batches, got):
                call(b, out, lse, ws)
    for _ in range(5):
        for out, lse in got:
            out.fill_(7.0)
            lse.fill_(7.0)
        g.replay()
        out, lse = empty()
        call(batches[2], out, lse, ws)
        torch.cuda.synchronize()
        assert torch.equal(out, want[2][0]) and native.dsa_sparse_attn_read_status(ws) == 0
        for pair, ref in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(pair, ref))
