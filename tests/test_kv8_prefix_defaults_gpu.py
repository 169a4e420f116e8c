"""The attention for requests that share prefixes with the parameters that dsa_kv8_params_init fills in."""

import numpy as np
import pytest
import torch

from oracle import paged
from test_kv8_prefix_gpu import PrefixCase, _lib  # noqa: F401
from top_sparse_mla_gb300 import native

pytestmark = pytest.mark.gpu


def test_a_batch_of_single_queries_costs_what_it_has():
    """max_q_len, by default n_tokens, says how many queries a request may have, not how many there are: 1500 requests of one
    query take about as long with it as with 1.  (Measured: 58 and 64 us; with CTAs for n_tokens
    queries of each request it took some ms.)"""
    c = PrefixCase(71, [(1, 130 + i % 20) for i in range(1500)], [(1500, 128)], page=16, h=1, g=8, d=128)
    D = c.device()
    times = {}
    for most in (1, None):
        p = native.dsa_kv8_params_init(D["q"], D["kp"], D["table"], max_q_len=most)
        ws = torch.empty(native.dsa_kv8_prefix_workspace_size(p, 1), dtype=torch.uint8, device="cuda")
        out, lse = torch.full_like(D["q"], 7.0), torch.full((c.n, 8), 7.0, device="cuda")
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        for i in range(12):
            if i == 2:
                a.record()
            native.dsa_kv8_prefix_attn_fwd(D["q"], D["kp"], D["vp"], D["ks"], D["vs"], D["table"], D["cu"], D["kv"], D["cug"], D["pre"], out,
                                           p, ws, lse=lse)
        b.record()
        assert native.dsa_sparse_attn_read_status(ws) == 0
        c.check(out, lse)
        times[most] = a.elapsed_time(b) * 100
    print(times)
    assert times[None] < 3 * times[1], times


@pytest.mark.parametrize("most", [19, 20, None], ids=["one skipped", "as many as there are", "default"])
def test_requests_of_few_queries_beside_one_of_many(most):
    # each row of the join looks for its request: requests without queries, of no group and skipped among them
    lens = [(0, 90)] + [(1, 300 + i) for i in range(40)] + [(0, 0), (20, 320), (0, 310)] + [(1, 64 + i) for i in range(9)] + [(0, 7)]
    c = PrefixCase(72, lens, [(1, None), (43, 288), (10, 48)], page=16, h=2, g=8, d=64)
    D = c.device()
    if most is None:
        most = c.n
    out, lse, status = c.run(D, max_q_len=most)
    ref = list(paged.kv8_attention(c.q.double().numpy(), c.kp, c.vp, c.ks, c.vs, c.table, c.cu, c.kv, float(np.float32(c.scale)), 0))
    if most == 19:
        ref[0][41:61], ref[1][41:61] = np.nan, np.nan
    assert status == (native.DSA_STATUS_QUERY_TOO_LONG if most == 19 else 0)
    c.check(out, lse, tuple(ref))
