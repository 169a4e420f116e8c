"""The attention over the paged 8-bit cache (include/dsa_kv8.h) where its kernels could go wrong: moves of the running
maximum, magnitudes and batch sizes at the ends of their ranges.  Case, its check and the error bound are those of
test_kv8_attn_gpu."""

import ctypes
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

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


def _batch(n):
    """n requests of up to two queries, a group of 2: all of them for rows_kernel."""
    rng = np.random.default_rng(n)
    return Case(n, [(int(a), int(b)) for a, b in zip(rng.integers(0, 3, n), rng.integers(0, 40, n))], h=1, g=2, d=64, page=16)


# 2783 requests are the first whose prefix sums and the plan's other shared memory pass 48 KB together; those of 4000 do so
# alone.  A kernel keeps a limit that was raised: each size in a process of its own.
@pytest.mark.parametrize("n", [2782, 2783, 3000, 4000, native.DSA_KV8_MAX_REQ])
def test_large_batches_as_a_process_first_call(n):
    code = f"import test_kv8_attn_edges_gpu as t; t._check(t._batch({n}))"
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([here, os.path.dirname(here), os.environ.get("PYTHONPATH", "")]))
    run = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]


def test_large_batches_from_several_host_threads():
    """The C calls of two batch sizes, each from two threads on streams of their own: a smaller batch's call lowered the limit of
    shared memory between a larger one's setting it and its launch, which refused one in a hundred of the larger ones."""
    lib = native.library()
    cases = [_batch(n) for n in (4000, native.DSA_KV8_MAX_REQ)]
    calls = []
    for c in cases + cases:
        D = c.device()
        p = native.dsa_kv8_params_init(D["q"], D["kp"], D["table"], max_q_len=2, softmax_scale=c.scale)
        out = torch.full((c.n, c.h * c.g, c.d), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((c.n, c.h * c.g), 7.0, device="cuda")
        ws = torch.empty(native.dsa_kv8_attn_workspace_size(p), dtype=torch.uint8, device="cuda")
        stream = torch.cuda.Stream()
        pitch = (c.h * c.g * c.d, c.d)
        args = (D["q"].data_ptr(), *pitch, *(D[x].data_ptr() for x in ("kp", "vp", "ks", "vs", "table")), D["table"].stride(0),
                D["cu"].data_ptr(), D["kv"].data_ptr(), out.data_ptr(), *pitch, lse.data_ptr(), ctypes.byref(p), ws.data_ptr(),
                ws.nbytes, stream.cuda_stream)
        calls.append((c, D, out, lse, ws, p, stream, args))
    torch.cuda.synchronize()
    failed = [0] * len(calls)

    def loop(i):
        stream, args = calls[i][-2:]
        for j in range(3000):
            failed[i] += lib.dsa_kv8_attn_fwd(*args) != native.DSA_OK
            if j % 16 == 15:
                stream.synchronize()

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert failed == [0] * len(calls)
    for c, _, out, lse, *_ in calls[:2]:
        c.check(out, lse)


ROWS, ONE_CTA, CLUSTER, MANY = [(1, 300), (2, 700)], [(40, 384)], [(40, 1280)], [(9, 640)] * 70


def _average(c):
    """Values of 1 to 2, of which every output, an average of some of them, has to be one as well (2^-7: the rounding of
    the weights to fp16 and of the result to bf16, 2^-11 + 2^-8 relative), and the logarithm of the sum of the weights has the
    scores' size."""
    values = np.random.default_rng(5).choice(np.arange(0x38, 0x41), c.vp.shape)   # the codes of 1, 1.125, .. 2
    c.vp[:] = values
    out, lse, status = c.run()
    assert status == 0
    a, b = int(c.cu[0]), int(c.cu[-1])
    got = out[a:b].double().cpu().numpy()
    low, high = got.min(), got.max()
    assert low >= 1 - 2.0 ** -7 and high <= 2 + 2.0 ** -6, (low, high)   # NaN fails both
    want = c.reference()[1][a:b]
    assert np.abs(lse[a:b].double().cpu().numpy() - want).max() <= 2.0 ** -18 * np.abs(want).max()


@pytest.mark.parametrize("lens", [ROWS, ONE_CTA, CLUSTER, MANY], ids=["rows", "one CTA", "cluster", "many tiles"])
@pytest.mark.parametrize("mag", [2.0 ** 27, 2.0 ** 29, 2.0 ** 31, 2.0 ** 40, 2.0 ** 90])
@pytest.mark.parametrize("kind", ["high", "low", "both"])
def test_scores_whose_steps_are_large(lens, mag, kind):
    """The steps between fp32 values of these scores are powers of two that a weight cannot hold."""
    c = _with_scores(81, lens, [-1.0 if kind == "low" else 1.0] * 1280, step_values=False, g=8, d=128, page=32)
    c.scale = 0.7
    c.q[:, :, 0] = mag
    if kind == "both":
        rng = np.random.default_rng(int(np.log2(mag)))
        c.kp[..., 0] = rng.integers(0x30, 0x38, c.kp.shape[:3]) + 0x80 * rng.integers(0, 2, c.kp.shape[:3])
    _average(c)


@pytest.mark.parametrize("lens", [ROWS, ONE_CTA, CLUSTER], ids=["rows", "one CTA", "cluster"])
def test_scores_far_below_zero(lens):
    # every score is -0.7e32
    c = _with_scores(80, lens, [-1.0] * 1280, step_values=False, g=8, d=128, page=32)
    c.scale = 0.7
    c.q[:, :, 0] = 1.0e32
    _average(c)


@pytest.mark.parametrize("lens", [ROWS, ONE_CTA, CLUSTER, [(1, 9000)]], ids=["rows", "one CTA", "cluster", "many CTAs"])
@pytest.mark.parametrize("scales", [[2.0 ** -64, 2.0 ** 64], [2.0 ** -63, 2.0 ** 40, 1.0, 2.0 ** 64], [2.0 ** -33, 2.0 ** -32, 2.0 ** 64],
                                    [2.0 ** -31, 2.0 ** 59], [2.0 ** -31, 2.0 ** 60]],
                         ids=["ends", "spread", "border", "below 2^90", "above 2^90"])
@pytest.mark.parametrize("d", [64, 128])
def test_value_scales_far_apart(lens, scales, d):
    """A token's share of the softmax's sum does not depend on its page's value scale."""
    _check(Case(82, lens, h=1, g=8, d=d, page=16, v_scale=scales, q_mag=0.5))


@pytest.mark.parametrize("lens", [ROWS, ONE_CTA, CLUSTER], ids=["rows", "one CTA", "cluster"])
def test_value_scales_that_rise_or_fall(lens):
    """Pages of the least scale, then of the largest, and the other way round: the sum is rescaled by 2^-128, or gains so little."""
    for order in (1, -1):
        c = Case(83, lens, h=1, g=8, d=128, page=16, poison=False, q_mag=0.5)
        for r, (_, kv) in enumerate(lens):
            for j in range(-(-kv // 16)):
                c.vs[c.table[r, j]] = 2.0 ** (64 * order * (1 if j >= kv // 32 else -1))
        _check(c)


@pytest.mark.parametrize("lens", [[(2, 700), (1, 300)] * 8, [(40, 700), (3, 1200)], [(33, 2100)], [(9, 640), (20, 700)] * 80],
                         ids=["rows", "tiles", "cluster", "many tiles"])
def test_value_scales_far_apart_under_a_window_and_in_some_requests(lens):
    """Every third request has value scales far apart: units with and without them follow one another."""
    c = Case(85, lens, h=2, g=8, d=64, page=32, window=333, poison=False, q_mag=0.5, v_scale=[1.0, 2.0])
    rng = np.random.default_rng(6)
    for r, (_, kv) in enumerate(lens):
        if r % 3 == 0:
            for j in range(-(-kv // 32)):
                c.vs[c.table[r, j]] = rng.choice(np.array([2.0 ** -64, 2.0 ** -40, 1.0, 2.0 ** 63], np.float32), 2)
    _check(c)


@pytest.mark.parametrize("lens", [ROWS, ONE_CTA, CLUSTER, MANY], ids=["rows", "one CTA", "cluster", "many tiles"])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_queries_that_are_not_finite_and_see_no_page(lens, what):
    """A row that sees nothing is 0 with an lse of -inf, whatever its query holds."""
    c = Case(84, lens, h=1, g=8, d=128, page=32)
    c.table[:] = -1
    c.q[:, ::3] = what
    _check(c)


@pytest.mark.parametrize("lens", [ROWS, ONE_CTA, CLUSTER, MANY], ids=["rows", "one CTA", "cluster", "many tiles"])
def test_queries_that_are_not_finite_leave_other_rows_alone(lens):
    """A row with a NaN that sees something is NaN, and the others are within the error bound."""
    c = Case(86, lens, h=1, g=8, d=128, page=32)
    c.q[:, 2::3, 5] = float("nan")
    out, lse, status = c.run()
    c.q[:, 2::3, 5] = 1.0
    want, want_lse, _ = c.run()
    assert status == 0
    a, b = int(c.cu[0]), int(c.cu[-1])
    assert out[a:b, 2::3].isnan().all() and lse[a:b, 2::3].isnan().all()
    out[a:b, 2::3], lse[a:b, 2::3] = want[a:b, 2::3], want_lse[a:b, 2::3]
    c.check(out, lse)


@pytest.mark.parametrize("lens,h", [([(1, 300), (1, 2000)], 2), ([(1, 20 + i) for i in range(9)], 8), ([(2, 700), (1, 5)], 1), ([(40, 90)], 2),
                                    ([(9, 200)] * 8, 2), ([(40, 90)] * 80, 1)])
@pytest.mark.parametrize("d,window", [(128, 0), (128, 100), (64, 0)])
def test_tables_far_wider_than_their_contexts(lens, h, d, window):
    """Room for 64k tokens a request, as an engine's tables have it: what the launches go by is the room."""
    _check(Case(98, lens, h=h, g=8, d=d, page=16, window=window, cols_more=4096))


@pytest.mark.parametrize("lens", [[(1, 300), (2, 0), (4, 90), (1, 17)], [(40, 300), (33, 0), (9, 128), (60, 90)], [(40, 1280), (1, 0)]],
                         ids=["rows", "tiles", "cluster"])
@pytest.mark.parametrize("window", [0, 50])
def test_lengths_outside_their_range_are_taken_as_the_nearest_bound(lens, window):
    c = Case(99, lens, h=1, g=8, d=64, page=16, window=window, poison=False, pad=0)
    room = c.table.shape[1] * c.page
    c.kv[0], c.kv[1] = room, 0
    D = c.device()
    want = c.run(dev=D)
    assert want[2] == 0
    far = dict(D, kv=D["kv"].clone(), cu=D["cu"].clone())
    far["kv"][0], far["kv"][1] = 2 ** 31 - 1, -2 ** 31
    far["cu"][-1] = 2 ** 31 - 1
    got = c.run(dev=far)
    assert got[2] == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c.check(*want[:2])
    # the first request's rows begin in front of the batch: they are those from row 0 on
    far["cu"][0], D["cu"][0] = -2 ** 31, 0
    most = max(q for q, _ in lens) + 1
    a, b = c.run(dev=far, max_q_len=most), c.run(dev=D, max_q_len=most)
    assert torch.equal(a[0][1:], b[0][1:]) and torch.equal(a[1][1:], b[1][1:])
