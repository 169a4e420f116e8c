"""The norm and rotation of heads (include/dsa_qk_norm_rope.h) against the oracle (oracle/heads.py) in float64.

Error bound of a value, with u = 2^-24, size = |a| + |b| of its rotary pair (derived before any run):
  - rounding of the result: half a step, 2^-8 |o| (bf16) or 2^-11 |o| (fp16); half of the smallest fp16 step, 2^-25;
  - the norm: the sum of squares is off by at most 13 u (eight products in a row, five levels), the mean and eps by
    2 u more, of which the root halves: 8 u, root and quotient 2 u, two products 2 u: 12 u of size;
  - the turn: its fraction is cut at 2^-24 of a turn, 2 pi 2^-24 < 7 u in the angle, cosine and sine 4 u of their own, products and sum 3 u:
    (7 + 4 + 3) u of size.
Together half |o| + 26 u size (1 % more for products of these terms)."""

import numpy as np
import pytest
import torch

from oracle import heads
from top_sparse_mla_gb300 import native

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"bf16": (torch.bfloat16, 2.0 ** -8), "fp16": (torch.float16, 2.0 ** -11)}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from top_sparse_mla_gb300.build import build
    build()
    native.library()


def _inputs(n, h_q, h_k, d, dtype, seed, pos=None, mag=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((n, h_q + 2 * h_k + 1, d), generator=g) * mag).to(TYPES[dtype][0])
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(TYPES[dtype][0]) for _ in range(2)]
    if pos is None:
        pos = torch.randint(0, 1 << 20, (n,), generator=g)
    return x, w, pos.to(torch.int32)


def _check(got, x, w, pos, dtype, **kw):
    want, size = heads.norm_rope(x.double().numpy(), None if w is None else w.double().numpy(), pos.numpy(), **kw)
    err = np.abs(got.double().cpu().numpy() - want)
    bound = TYPES[dtype][1] * np.abs(want) + 26 * 1.01 * U * size + 2.0 ** -25
    assert (err <= bound).all(), f"{(err > bound).sum()} of {err.size}, worst {np.max(err / bound)} of the bound"


def _call(x, w, pos, h_q, h_k, norm=(True, True), q_out=None, k_out=None, stream=None, **kw):
    xd, pd = x.cuda(), pos.cuda()
    n, _, d = x.shape
    q, k = xd[:, :h_q], xd[:, h_q:h_q + h_k] if h_k else None
    qo = torch.full((n, h_q, d), 7.0, dtype=x.dtype, device="cuda")
    ko = torch.full((n, h_k, d), 7.0, dtype=x.dtype, device="cuda") if h_k else None
    p = native.dsa_qk_params_init(q, k, **kw)
    native.dsa_qk_norm_rope(q, k, pd, w[0].cuda() if norm[0] else None, w[1].cuda() if norm[1] and h_k else None, qo, ko, p)
    torch.cuda.synchronize()
    assert torch.equal(xd.cpu().view(torch.int16), x.view(torch.int16)), "the inputs were written"
    return qo, ko


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n,h_q,h_k,d,rot,start,inter", [
    (1, 1, 0, 64, 64, 0, False), (3, 5, 1, 128, 128, 0, False), (2, 8, 8, 128, 64, 64, True), (7, 4, 2, 192, 64, 128, True),
    (5, 3, 3, 256, 256, 0, False), (4, 6, 2, 256, 128, 128, False), (33, 2, 1, 80, 32, 8, False), (9, 7, 1, 112, 96, 16, True),
    (130, 1, 0, 64, 64, 0, True), (300, 1, 1, 144, 16, 120, False), (2, 64, 8, 128, 0, 0, False), (41, 12, 2, 192, 192, 0, False),
    (17, 1, 16, 240, 224, 8, True)])
def test_shapes(n, h_q, h_k, d, rot, start, inter, dtype):
    x, w, pos = _inputs(n, h_q, h_k, d, dtype, n + d)
    kw = dict(rotary_dim=rot, rotary_start=start, interleaved=inter)
    for norm in ((True, True), (False, False), (True, False), (False, True)):
        q, k = _call(x, w, pos, h_q, h_k, norm, **kw)
        _check(q, x[:, :h_q], w[0] if norm[0] else None, pos, dtype, **kw)
        if h_k:
            _check(k, x[:, h_q:h_q + h_k], w[1] if norm[1] else None, pos, dtype, **kw)


def test_many_tokens_and_heads():
    # more rows than CTAs at once, and CTAs that begin inside a token
    for n, h_q, h_k in ((700, 13, 3), (5000, 1, 0), (12, 500, 100)):
        x, w, pos = _inputs(n, h_q, h_k, 64, "bf16", n)
        q, k = _call(x, w, pos, h_q, h_k)
        _check(q, x[:, :h_q], w[0], pos, "bf16", rotary_dim=64)
        if h_k:
            _check(k, x[:, h_q:h_q + h_k], w[1], pos, "bf16", rotary_dim=64)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("base", [10000.0, 500000.0, 1.0, 0.5])
def test_positions_and_bases(inter, base):
    # the oracle's own product of position and frequency is off by 2^-53 of up to 2^24 radians (2^31 for base 0.5's 16 pairs)
    pos = torch.tensor([0, 1, -1, 17, -4096, 1 << 20, (1 << 24) + 1, -(1 << 24)])
    x, w, pos = _inputs(len(pos), 2, 1, 64, "fp16", 5, pos)
    q, _ = _call(x, w, pos, 2, 1, rotary_dim=32, interleaved=inter, rope_base=base)
    _check(q, x[:, :2], w[0], pos, "fp16", rotary_dim=32, interleaved=inter, base=base)


@pytest.mark.parametrize("mag", [2.0 ** -60, 1e-3, 2.0 ** 60])
def test_magnitudes(mag):
    x, w, pos = _inputs(6, 3, 1, 128, "bf16", 6, mag=mag)
    for eps in (1e-6, 0.0):
        q, _ = _call(x, w, pos, 3, 1, rms_eps=eps)
        _check(q, x[:, :3], w[0], pos, "bf16", rotary_dim=128, eps=float(np.float32(eps))) if mag > 1e-10 or eps > 0 else None
    x[0] = 0
    q, k = _call(x, w, pos, 3, 1)
    assert (q[0] == 0).all() and (k[0] == 0).all()


def test_values_that_are_not_finite_stay_in_their_row():
    x, w, pos = _inputs(4, 3, 1, 128, "bf16", 8)
    good, _ = _call(x, w, pos, 3, 1)
    x[1, 1, 5], x[2, 0, 7] = float("nan"), float("inf")
    q, _ = _call(x, w, pos, 3, 1)
    assert q[1, 1].isnan().all()
    keep = torch.ones((4, 3), dtype=torch.bool)
    keep[1, 1] = keep[2, 0] = False
    assert torch.equal(q[keep.cuda()], good[keep.cuda()])


def test_in_place_and_other_layouts():
    n, h_q, h_k, d = 19, 4, 2, 128
    x, w, pos = _inputs(n, h_q, h_k, d, "bf16", 9)
    want_q, want_k = _call(x, w, pos, h_q, h_k)
    y = x.cuda()
    q, k = y[:, :h_q], y[:, h_q:h_q + h_k]
    p = native.dsa_qk_params_init(q, k)
    args = pos.cuda(), w[0].cuda(), w[1].cuda()
    native.dsa_qk_norm_rope(q, k, *args, q, k, p)
    assert torch.equal(q, want_q) and torch.equal(k, want_k) and torch.equal(y[:, h_q + h_k:].cpu(), x[:, h_q + h_k:])
    # heads outermost, in and out
    z = x.cuda()[:, :h_q].transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.zeros((h_q, n + 3, d), dtype=x.dtype, device="cuda")
    native.dsa_qk_norm_rope(z, None, args[0], args[1], None, out[:, 1:n + 1].transpose(0, 1), None, native.dsa_qk_params_init(z))
    assert torch.equal(out[:, 1:n + 1].transpose(0, 1), want_q) and (out[:, 0] == 0).all() and (out[:, n + 1:] == 0).all()
    # another base between two calls of the same shape, and back
    _check(_call(x, w, pos, h_q, h_k, rope_base=500.0)[0], x[:, :h_q], w[0], pos, "bf16", rotary_dim=d, base=500.0)
    assert torch.equal(_call(x, w, pos, h_q, h_k)[0], want_q)


def test_empty_graph_and_other_stream():
    x, w, pos = _inputs(21, 8, 2, 128, "fp16", 10)
    want, _ = _call(x, w, pos, 8, 2)
    empty = torch.empty((0, 8, 128), dtype=torch.float16, device="cuda")
    native.dsa_qk_norm_rope(empty, None, torch.empty(0, dtype=torch.int32, device="cuda"), None, None, empty, None,
                            native.dsa_qk_params_init(empty))
    xd, pd, wd = x.cuda(), pos.cuda(), [a.cuda() for a in w]
    q, k = xd[:, :8], xd[:, 8:10]
    qo, ko = torch.empty_like(q.contiguous()), torch.empty_like(k.contiguous())
    p = native.dsa_qk_params_init(q, k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            native.dsa_qk_norm_rope(q, k, pd, *wd, qo, ko, p)
    xd.copy_(xd.flip(0))
    pd.copy_(pd.flip(0))
    qo.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(qo.flip(0), want)
