"""Latent attention in its expanded form (include/dsa_mla_prefill.h) on batches of more than 256 tiles, 512 and 1024 requests, whose
plan is the one of 1024 threads.  Cases, oracle and error bound are those of test_mla_prefill_gpu.py."""

import pytest

from test_mla_prefill_gpu import SPLIT, WHOLE, Case, _check, _lib  # noqa: F401
from top_sparse_mla_gb300 import native

pytestmark = pytest.mark.gpu

# units may be split whatever their number, up to 1024 tiles: none is expected
FEW = {"max_q_len": 0, "max_kv_len": 1 << 20}


@pytest.mark.parametrize("how", [SPLIT, WHOLE], ids=["split", "whole"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_more_than_256_tiles(how, dtype):
    # room for 264 tiles: more than 256, and fewer than two an SM
    _check(Case(81, [(120 + i, 120 + i + 37 * (i % 7)) for i in range(90)] + [(1 + i % 3, 300 + i) for i in range(104)] + [(270, 900)] * 6, h=1,
                dtype=dtype), **how)


@pytest.mark.parametrize("how", [SPLIT, WHOLE], ids=["split", "whole"])
def test_a_prompt_of_more_than_65_thousand_queries(how):
    # 274 tiles of one request, of which the last rows alone see keys
    _check(Case(82, [(2, 700), (70000, 40), (3, 300)], h=1), **how)


@pytest.mark.parametrize("n", [513, 700, 1025, 1500])
def test_many_requests(n):
    _check(Case(83, [(1 + i % 3, 1 + i % 3 + i % 41) for i in range(n)], h=2))
    _check(Case(84, [(i % 2, 1 + i % 300) for i in range(n)], h=1, dtype="fp16"), **FEW)


def test_many_requests_few_of_which_have_queries():
    _check(Case(85, [(5 if i % 97 == 3 else 0, 400 if i % 97 == 3 else i % 4) for i in range(1000)], h=3), **FEW)


def test_as_many_requests_as_there_may_be():
    _check(Case(86, [(1, 1 + i % 5) for i in range(native.DSA_MLA_MAX_REQ)], h=1))


def test_more_queries_than_were_said():
    # tiles beyond those that the choice went by
    c = Case(87, [(300, 700)] * 3 + [(20, 90)] * 400, h=1)
    _check(c, **FEW)
    _check(c, max_q_len=1, max_kv_len=0)
