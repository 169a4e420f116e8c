"""The failure path of the attention over the paged 8-bit cache, without a GPU fault: an on-chip wait that runs out.

DSA_KV8_FLAG_TEST_WAIT_TIMEOUT makes CTA 0's copies stop after three blocks, with products and copies under way, and wait for
what nothing completes.  That wait gives up after about a second, the call's status says so, and all roles of the CTA stop.  The
rows of the other CTAs are bit for bit those of a clean call, and so is everything in the next call."""

import time

import pytest
import torch

from test_kv8_attn_gpu import TYPES, Case
from top_sparse_mla_gb300 import native

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from top_sparse_mla_gb300.build import build
    build()
    native.library()


def _run(c, D, ws, flags=0):
    out = torch.full((c.n, c.h * c.g, c.d), 7.0, dtype=TYPES[c.dtype][0], device="cuda")
    lse = torch.full((c.n, c.h * c.g), 7.0, device="cuda")
    p = native.dsa_kv8_params_init(D["q"], D["kp"], D["table"], max_q_len=max(q for q, _ in c.lens), softmax_scale=c.scale, flags=flags)
    if ws is None:
        ws = torch.empty(native.dsa_kv8_attn_workspace_size(p), dtype=torch.uint8, device="cuda")
    t0 = time.perf_counter()
    native.dsa_kv8_attn_fwd(D["q"], D["kp"], D["vp"], D["ks"], D["vs"], D["table"], D["cu"], D["kv"], out, p, ws, lse=lse)
    return out, lse, native.dsa_sparse_attn_read_status(ws), ws, time.perf_counter() - t0


@pytest.mark.parametrize("lens,h,split", [([(20, 700)] * 90, 2, False), ([(40, 9000)], 4, True), ([(33, 9000), (70, 8000)], 2, True)],
                         ids=["a CTA for each tile", "clusters", "clusters and a half without rows"])
@pytest.mark.parametrize("d", [64, 128])
def test_a_wait_that_runs_out_is_reported_and_recovered_from(lens, h, split, d):
    c = Case(95, lens, h=h, g=8, d=d, page=32)
    D = c.device()
    want, want_lse, status, ws, _ = _run(c, D, None)
    assert status == 0
    out, lse, status, _, seconds = _run(c, D, ws, native.DSA_KV8_FLAG_TEST_WAIT_TIMEOUT)
    assert status == native.DSA_STATUS_WAIT_TIMEOUT
    assert 0.3 < seconds < 20.0, seconds
    same = (out == want).all(dim=-1) & (lse == want_lse)
    a, b = int(c.cu[0]), int(c.cu[-1])
    if split:
        # a cluster's unit is one tile and KV head: all other heads' rows, and at most 256 rows of one head
        wrong = (~same[a:b]).nonzero()
        assert len(wrong) <= 256 and len((wrong[:, 1] // c.g).unique()) <= 1
    else:
        # a CTA's units are one or two of the 180 tiles of 160 rows, unwritten
        unwritten = (out == 7.0).all(dim=-1) & (lse == 7.0)
        assert (same | unwritten)[a:b].all() and 0 < int(unwritten[a:b].sum()) <= 2 * 160
    out, lse, status, _, _ = _run(c, D, ws)
    assert status == 0 and torch.equal(out, want) and torch.equal(lse, want_lse)


def test_without_tiles_the_flag_changes_nothing():
    c = Case(96, [(1, 700), (2, 90)], h=2, g=8, d=128, page=32)
    D = c.device()
    want, want_lse, _, ws, _ = _run(c, D, None)
    out, lse, status, _, _ = _run(c, D, ws, native.DSA_KV8_FLAG_TEST_WAIT_TIMEOUT)
    assert status == 0 and torch.equal(out, want) and torch.equal(lse, want_lse)
