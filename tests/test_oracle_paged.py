"""Pins of the paged-cache oracle (oracle/paged.py), CPU only: hand-worked maps, closed
forms of the insert's scales and codes, and the attention against a scalar restatement."""

import math

import numpy as np
import pytest

from oracle import codecs, paged


def test_page_map_hand_worked():
    # pages of 4: request 0 has 3 tokens in page 9 and adds 2, request 1 adds 5, request 2 nothing
    table = np.array([[9, -7, -7], [-7, -7, -7], [3, -7, -7]], np.int32)
    got = paged.page_map([3, 0, 2], [2, 5, 0], table, [20, 21, 22, 23], 4, 9)
    t, cu, kv, pos, slots, req, info = got
    assert t.tolist() == [[9, 20, -7], [21, 22, -7], [3, -7, -7]]
    assert cu.tolist() == [0, 2, 7, 7] and kv.tolist() == [5, 5, 2]
    assert pos.tolist() == [3, 4, 0, 1, 2, 3, 4, 0, 0]
    assert slots.tolist() == [39, 80, 84, 85, 86, 87, 88, -1, -1]
    assert req.tolist() == [0, 0, 1, 1, 1, 1, 1, -1, -1] and info.tolist() == [3, 0]


def test_page_map_reports_what_does_not_fit():
    table = np.full((2, 2), -1, np.int32)
    t, cu, kv, pos, slots, _, info = paged.page_map([0, 0], [4, 9], table, [5, 6], 4, 12)
    assert info.tolist() == [2, paged.OUT_OF_PAGES | paged.TABLE_FULL | paged.TOKENS_FULL]
    assert t.tolist() == [[5, -1], [6, -1]] and cu.tolist() == [0, 4, 12] and kv.tolist() == [4, 9]
    assert slots.tolist() == [20, 21, 22, 23, 24, 25, 26, 27, -1, -1, -1, -1]
    assert pos.tolist() == [0, 1, 2, 3, 0, 1, 2, 3, 4, 5, 6, 7]


@pytest.mark.parametrize("amax,s", [(0.0, 2.0 ** -64), (448.0, 1.0), (448.0001, 2.0), (224.0, 0.5), (1.0, 2.0 ** -8),
                                    (1e-30, 2.0 ** -64), (1e30, 2.0 ** 64), (1.75, 2.0 ** -8), (1.76, 2.0 ** -7)])
def test_page_scale(amax, s):
    assert paged.page_scale(amax) == s


def test_insert_codes_do_not_depend_on_how_a_page_was_filled():
    # values of at least 2^-6 of the final scale: every split of the page's tokens gives the same page
    rng = np.random.default_rng(0)
    x = np.sign(rng.standard_normal((16, 2, 4))) * rng.uniform(0.5, 100.0, (16, 2, 4))
    slots = 16 + np.arange(16)
    want = None
    for cuts in ([0, 16], [0, 1, 2, 16], [0, 5, 11, 16], list(range(17))):
        pool, scale = np.full((3, 2, 16, 4), 0x55, np.uint8), np.full((3, 2), 3.0, np.float32)
        for a, b in zip(cuts[:-1], cuts[1:]):
            pool, scale = paged.kv8_insert(pool, scale, x[a:b], slots[a:b])
        assert (pool[[0, 2]] == 0x55).all() and (scale[[0, 2]] == 3.0).all()
        v = codecs.e4m3_decode(pool[1]) * scale[1][:, None, None]
        assert np.max(np.abs(v - x.transpose(1, 0, 2)) / np.abs(x.transpose(1, 0, 2))) <= 2.0 ** -4
        want = (pool, scale) if want is None else want
        assert np.array_equal(pool, want[0]) and np.array_equal(scale, want[1])


def test_attention_against_scalars():
    rng = np.random.default_rng(1)
    n_pages, h, page, d, g = 5, 2, 4, 3, 2
    kp, vp = (codecs.e4m3_encode(rng.standard_normal((n_pages, h, page, d)) * 20) for _ in range(2))
    ks, vs = (rng.uniform(0.01, 0.1, (n_pages, h)).astype(np.float32) for _ in range(2))
    table = np.array([[3, 1, -1], [0, 9, 2], [4, -1, -1]], np.int32)   # 9: no such page
    cu, kv = [1, 4, 6, 6], [6, 11, 3]
    q = rng.standard_normal((8, h * g, d))
    for window in (0, 1, 3):
        out, lse, _ = paged.kv8_attention(q, kp, vp, ks, vs, table, cu, kv, 0.7, window)
        for t in range(8):
            r = 0 if 1 <= t < 4 else 1 if 4 <= t < 6 else None
            for head in range(h * g):
                if r is None:
                    assert np.isnan(out[t, head]).all() and math.isnan(lse[t, head])
                    continue
                p, hh = kv[r] - (cu[r + 1] - cu[r]) + t - cu[r], head // g
                num, den = [0.0] * d, 0.0
                for j in range(p + 1):
                    pg = int(table[r, j // page])
                    if (window and j <= p - window) or not 0 <= pg < n_pages:
                        continue
                    kk = codecs.e4m3_decode(kp[pg, hh, j % page]) * float(ks[pg, hh])
                    vv = codecs.e4m3_decode(vp[pg, hh, j % page]) * float(vs[pg, hh])
                    e = math.exp(0.7 * sum(float(kk[i]) * q[t, head, i] for i in range(d)))
                    den += e
                    num = [a + e * float(b) for a, b in zip(num, vv)]
                if den == 0.0:
                    assert (out[t, head] == 0).all() and lse[t, head] == -math.inf
                else:
                    assert np.allclose(out[t, head], np.array(num) / den, rtol=1e-12, atol=1e-14)
                    assert abs(lse[t, head] - math.log(den)) < 1e-12
