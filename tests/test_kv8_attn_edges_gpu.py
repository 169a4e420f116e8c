"""The attention over the paged 8-bit cache (include/dsa_kv8.h) where its kernels could go wrong: moves of the running
maximum, magnitudes and batch sizes at the ends of their ranges.  Case, its check and the error bound are those of
test_kv8_attn_gpu."""

import numpy as np
import pytest

from oracle import codecs
from test_kv8_attn_gpu import Case, _check
from top_sparse_mla_gb300 import native

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from top_sparse_mla_gb300.build import build
    build()
    native.library()


def _with_scores(seed, lens, scores, step_values=True, **kw):
    """A case in which every query's score of cached token j is scores[j] * ln 2, for every request.  With step_values, a
    token whose score is the largest so far has zeros in the odd dims of its value, where the tokens before it show."""
    c = Case(seed, lens, h=1, v_scale=[1.0], poison=False, scale=float(np.log(2.0)), **kw)
    c.ks[:] = 1.0
    c.q[:] = 0.0
    c.q[:, :, 0] = 1.0
    c.kp[:] = 0
    code = codecs.e4m3_encode(np.asarray(scores, np.float64))
    for r, (_, kv) in enumerate(lens):
        top = -np.inf
        for j in range(kv):
            page, row = c.table[r, j // c.page], j % c.page
            c.kp[page, 0, row, 0] = code[j]
            if step_values and scores[j] > top:
                c.vp[page, 0, row, 1::2] = 0
                top = scores[j]
    return c


@pytest.mark.parametrize("rise", [16, 20, 24])
@pytest.mark.parametrize("lens", [[(40, 384)], [(40, 1280)], [(9, 640)] * 70], ids=["one CTA", "cluster", "many tiles"])
@pytest.mark.parametrize("d", [64, 128])
def test_maxima_that_move_in_both_parts_of_a_block(rise, lens, d):
    """The largest score grows by `rise` at a token in each half of the third block of 128 and in each half of the last: the sums
    so far and the half block's weights are rescaled, and rescaled again at once.  In the odd dims the values are those of the
    tokens in front of the last rise."""
    kv = lens[0][1]
    scores, best = np.zeros(kv), 0
    for at in (256 + 5, 256 + 64 + 17) + ((kv - 128 + 9, kv - 64 + 30) if kv > 384 else ()):
        best += rise
        scores[at:] = best - 3
        scores[at] = best
    _check(_with_scores(rise + d, lens, scores, g=8, d=d, page=32))
