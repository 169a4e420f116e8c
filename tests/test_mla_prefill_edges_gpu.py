"""Latent attention in its expanded form (include/dsa_mla_prefill.h) where tests of the ordinary do not come.  Cases, oracle and error
bound are those of test_mla_prefill_gpu.py."""

import pytest
import torch

from test_mla_prefill_gpu import SPLIT, WHOLE, Case, _check, _lib  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("how", [SPLIT, WHOLE], ids=["split", "whole"])
@pytest.mark.parametrize("lens,rows", [
    ([(1, 1)], [0]),                                   # a prompt's first token: one score, of -inf
    ([(3, 3), (130, 400)], [0, 2, 3, 100, 132]),       # tiles of one half and of two
    ([(5, 3000)], [0, 4]),                             # a unit in many pieces, each without a weight
    ([(5, 3), (2, 0)], [0, 1, 2, 4, 5]),               # rows 0, 1 and 5 see nothing
], ids=str)
def test_a_query_whose_every_score_is_minus_infinity_spoils_its_row(lens, rows, how, dtype):
    c = Case(51, lens, dtype=dtype)
    c.up[3:c.m - 2, :, 7] = c.up[3:c.m - 2, :, 7].abs() + 0.01   # a dim of the keys that is positive everywhere
    want, want_l = _check(c, **how)
    keep = torch.ones_like(want_l, dtype=torch.bool)
    for r in rows:
        c.q[1 + r, 1, 7] = -float("inf")
        keep[1 + r, 1] = False
    out, lse, status = c.run(**how)
    assert status == 0
    assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], want_l[keep])
    empty = torch.isneginf(want_l)
    assert out[~keep & ~empty].isnan().all() and lse[~keep & ~empty].isnan().all()
    assert (out[~keep & empty] == 0).all() and torch.isneginf(lse[~keep & empty]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("how", [SPLIT, WHOLE], ids=["split", "whole"])
def test_a_row_with_one_key_has_its_value_as_it_is(how, dtype):
    # its weight is 1, whatever its score
    lens = [(1, 1)] * 40 + [(3, 3), (130, 130), (300, 300), (2, 1), (1, 700)]
    c = Case(52, lens, h=3, dtype=dtype)
    out, lse = _check(c, **how)
    v = c.up[:, :, 128:].cuda()
    for r, (ql, kv) in enumerate(lens[:-1]):
        row, key = int(c.cu[r]) + ql - kv, int(c.ck[r])
        assert torch.equal(out[row], v[key]), r
