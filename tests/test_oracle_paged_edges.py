"""Pins of the paged-cache oracle (oracle/paged.py) for values that are not finite, CPU only."""

import numpy as np
import pytest

from oracle import codecs, paged


@pytest.mark.parametrize("what,code", [(np.inf, 0x7E), (-np.inf, 0xFE), (np.nan, 0x7F)])
def test_values_that_are_not_finite_do_not_change_their_page_s_scale(what, code):
    pool = codecs.e4m3_encode(np.full((1, 1, 16, 4), 100.0))
    scale = np.full((1, 1), 2.0 ** -3, np.float32)
    x = np.full((2, 1, 4), 30.0)
    x[1, 0, 2] = what
    got, s = paged.kv8_insert(pool, scale, x, np.array([5, 6]))
    want, ws = paged.kv8_insert(pool, scale, np.full((2, 1, 4), 30.0), np.array([5, 6]))
    assert s[0, 0] == ws[0, 0] == 2.0 ** -3
    assert got[0, 0, 6, 2] == code
    want[0, 0, 6, 2] = code
    assert np.array_equal(got, want)
    # a run of nothing else: the least scale
    got, s = paged.kv8_insert(pool, scale, np.full((1, 1, 4), what), np.array([0]))
    assert s[0, 0] == 2.0 ** -64 and (got[0, 0, 0] == code).all()
