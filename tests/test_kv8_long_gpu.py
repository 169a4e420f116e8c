"""An attention call over the paged 8-bit cache that takes longer than its waits' limit, and is right."""

import numpy as np
import pytest
import torch

from test_kv8_attn_gpu import Case
from top_sparse_mla_gb300 import native

pytestmark = pytest.mark.gpu


def test_a_half_of_a_tile_that_has_nothing_to_do_for_long():
    """1400 requests of one query with 64 heads to a KV head, half a tile each, on 8 M tokens that share their pages, and a
    request of four queries and a short context, whose tile comes last: the other half's threads wait through all of it
    (some 12 s)."""
    c = Case(90, [(4, 300)], h=14, g=64, d=64, page=128)
    D = c.device()
    n, cols = 1400, 1 << 16
    first = int(c.cu[0])
    live = [int(x) for x in c.table[0, :2]]   # two full pages of the request's own
    table = torch.full((n + 1, cols), live[0], dtype=torch.int32, device="cuda")
    table[:, 1::2] = live[1]
    table[0, :c.table.shape[1]] = D["table"][0]
    end = int(c.cu[1])
    cu = torch.cat([D["cu"], torch.arange(end + 1, end + n + 1, dtype=torch.int32, device="cuda")])
    kv = torch.cat([D["kv"], torch.full((n,), cols * 128, dtype=torch.int32, device="cuda")])
    q = torch.ones((end + n, c.h * c.g, c.d), dtype=torch.bfloat16, device="cuda")
    q[first:end] = D["q"][first:end]
    out, lse = torch.full_like(q, 7.0), torch.full((end + n, c.h * c.g), 7.0, device="cuda")
    p = native.dsa_kv8_params_init(q, D["kp"], table, max_q_len=4, softmax_scale=c.scale)
    ws = torch.empty(native.dsa_kv8_attn_workspace_size(p), dtype=torch.uint8, device="cuda")
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    native.dsa_kv8_attn_fwd(q, D["kp"], D["vp"], D["ks"], D["vs"], table, cu, kv, out, p, ws, lse=lse)
    b.record()
    assert native.dsa_sparse_attn_read_status(ws) == 0, f"after {a.elapsed_time(b):.0f} ms"
    print(f"{a.elapsed_time(b):.0f} ms")
    assert bool(out[end:].isfinite().all())
    padded = torch.full((c.n, c.h * c.g, c.d), 7.0, dtype=torch.bfloat16, device="cuda")
    padded_lse = torch.full((c.n, c.h * c.g), 7.0, device="cuda")
    padded[first:end], padded_lse[first:end] = out[first:end], lse[first:end]
    c.check(padded, padded_lse)
    # the others are alike: two full pages over and over
    assert torch.equal(out[end:], out[end:end + 1].expand(n, -1, -1))
    assert np.allclose(lse[end, 0].item(), _lse(c, live), atol=1e-3)


def _lse(c, live):
    from oracle import codecs
    k = np.concatenate([codecs.e4m3_decode(c.kp[x, 0]) * float(c.ks[x, 0]) for x in live])
    z = k.sum(axis=1) * c.scale
    return z.max() + np.log(np.exp(z - z.max()).sum()) + np.log(2 ** 15)
