"""The attention for requests that share prefixes behind a context as long as positions can be."""

import pytest
import torch

from test_kv8_prefix_gpu import PrefixCase, _lib  # noqa: F401
from top_sparse_mla_gb300 import native

pytestmark = pytest.mark.gpu


def test_positions_of_a_group_stay_below_two_to_the_31():
    """Three prompt chunks of 620 queries behind 2^31 - 1024 tokens, of which only the first 512 and the last 1000 have pages: the
    group's rows, counted on from the last token that it shares, would pass 2^31.  The result is that of the tokens that are there,
    without the gap (some 2 s)."""
    page, cols, head = 128, (1 << 24) - 8, 4
    c = PrefixCase(41, [(620, 1499), (620, 1488), (620, 1477)], [(3, 1 << 30)], page=page, h=1, g=1, d=64)
    D = c.device()
    pages = 12
    gap = cols - pages
    table = torch.full((3, cols), -1, dtype=torch.int32, device="cuda")
    table[:, :head] = D["table"][:, :head]
    table[:, head + gap:] = D["table"][:, head:pages]
    kv, pre = D["kv"] + gap * page, torch.tensor([2 ** 31 - 1], dtype=torch.int32, device="cuda")
    out, lse = torch.full_like(D["q"], 7.0), torch.full((c.n, 1), 7.0, device="cuda")
    p = native.dsa_kv8_params_init(D["q"], D["kp"], table, max_q_len=620, softmax_scale=c.scale)
    ws = torch.full((native.dsa_kv8_prefix_workspace_size(p, 1),), 0xAB, dtype=torch.uint8, device="cuda")
    native.dsa_kv8_prefix_attn_fwd(D["q"], D["kp"], D["vp"], D["ks"], D["vs"], table, D["cu"], kv, D["cug"], pre, out, p, ws, lse=lse)
    assert native.dsa_sparse_attn_read_status(ws) == 0
    c.check(out, lse)
