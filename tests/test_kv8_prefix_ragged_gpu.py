"""The attention for requests that share prefixes (include/dsa_kv8_prefix.h) where the prefixes of a batch, and the tiles that come of
them, are of very unlike lengths: a short tile takes a CTA whatever its part of the blocks.  Cases, oracle and error bound are those of
test_kv8_prefix_gpu.py; tests/test_kv8_cuts_host.py has the cuts themselves."""

import pytest

from test_kv8_prefix_gpu import PrefixCase, _check, _lib  # noqa: F401

pytestmark = pytest.mark.gpu


def _groups(*prefixes, n=2, own=9):
    """n requests with one query each behind each prefix."""
    return [(1, p + 1 + own * i) for p in prefixes for i in range(n)], [(n, p) for p in prefixes]


@pytest.mark.parametrize("prefixes,d,page,dtype", [
    ((16384, 256, 256), 64, 64, "bf16"), ((256, 256, 16384), 64, 64, "fp16"), ((8192, 128, 128), 128, 16, "bf16"),
    ((128, 128, 8192), 64, 16, "bf16"), ((16, 8192, 16, 16, 16, 16, 16, 16), 64, 16, "bf16"), ((8192, 512, 512, 512, 512), 64, 128, "fp16")])
def test_prefixes_of_very_unlike_lengths(prefixes, d, page, dtype):
    lens, groups = _groups(*prefixes)
    _check(PrefixCase(31, lens, groups, page=page, h=8, g=8, d=d, dtype=dtype))


@pytest.mark.parametrize("first", [True, False], ids=["prompt first", "prompt last"])
def test_a_group_beside_a_prompt_of_no_group(first):
    lens, groups = _groups(8192)
    lens, groups = ([(200, 200)] + lens, [(1, None)] + groups) if first else (lens + [(200, 200)], groups + [(1, None)])
    _check(PrefixCase(32, lens, groups, page=64, h=8, g=8, d=64))


@pytest.mark.parametrize("h,n", [(1, 125), (2, 48)])
def test_a_long_prefix_beside_many_tiles_of_one_block(h, n):
    # all of them together are more than there are CTAs
    lens, groups = _groups(8192, n=5)
    short = [(5, 20 + i % 30) for i in range(n)]
    _check(PrefixCase(33, short + lens, [(n, None)] + groups, page=16, h=h, g=8, d=64))
    _check(PrefixCase(34, lens + short, groups + [(n, None)], page=16, h=h, g=8, d=128, dtype="fp16"))
