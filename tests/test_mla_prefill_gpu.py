"""Latent attention in its expanded form (include/dsa_mla_prefill.h) against the oracle (oracle/heads.py) in float64.

Error bound of an output value o = sum_j p_j v_j (derived from the stated numerics, before any run), with u = 2^-24:
  - rounding of the result: half a step, h |o| with h = 2^-8 (bf16) or 2^-11 (fp16), and half of fp16's smallest step, 2^-25;
  - each score has an error of at most delta: 192 products summed in fp32 in any order, then four more roundings, and the
    maximum's own size in the exponent: delta <= 200 u size + 8 u (|lse| + size), size = max_j sum_i |q_i k_ij| softmax_scale;
    the exponential adds 2^-21 relative.  A relative error eps of every weight changes o by at most 2 eps mass,
    mass = sum_j p_j |v_j|;
  - the weights' rounding for the product: h mass, and (fp16) half of the smallest step, 2^-25, of the subnormal ones, against a
    largest weight of at least 1: 2^-25 sum_j |v_j| max p <= 2^-25 n max |v|;
  - the fp32 sums over the n keys: n u mass.
lse: delta + 2^-21 + (n + 8) u + 2 u |lse|."""

import time

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


class Case:
    """lens: (q_len, kv_len) of each request.  Rows of no request, and keys that no query sees, are NaN."""

    def __init__(self, seed, lens, h=2, dtype="bf16", q_mag=1.5, scale=None, pad=2, gap=True):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.h, self.dtype = lens, h, dtype
        self.scale = 192 ** -0.5 if scale is None else scale
        self.cu = np.concatenate([[1], 1 + np.cumsum([a for a, _ in lens])]).astype(np.int32)
        self.ck = np.concatenate([[3], 3 + np.cumsum([b for _, b in lens])]).astype(np.int32)
        self.n, self.m = int(self.cu[-1]) + pad, int(self.ck[-1]) + pad
        t = TYPES[dtype][0]
        self.q = (torch.randn((self.n, h, 192), generator=g) * q_mag).to(t)
        self.up = torch.randn((self.m, h, 256), generator=g).to(t)        # keys and values side by side
        self.latent = torch.randn((self.m, 576), generator=g).to(t)       # the rotary keys inside the latent rows
        nan = float("nan")
        self.q[0] = nan
        self.q[self.n - pad:] = nan
        for x in (self.up, self.latent):
            x[:3] = nan
            x[self.m - pad:] = nan

    def device(self):
        t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        up, latent = self.up.cuda(), self.latent.cuda()
        return {"q": self.q.cuda(), "k": up[:, :, :128], "v": up[:, :, 128:], "r": latent[:, 512:], "cu": t(self.cu), "ck": t(self.ck)}

    def params(self, D, **kw):
        kw = {"max_q_len": max([a for a, _ in self.lens] + [0]), "max_kv_len": max([b for _, b in self.lens] + [0]),
              "softmax_scale": self.scale, **kw}
        return native.dsa_mla_params_init(D["q"], D["k"], D["cu"], **kw)

    def run(self, D=None, out=None, workspace=None, **kw):
        D = D or self.device()
        if out is None:
            out = torch.full((self.n, self.h, 128), 7.0, dtype=TYPES[self.dtype][0], device="cuda")
        lse = torch.full((self.n, self.h), 7.0, device="cuda")
        p = self.params(D, **kw)
        if workspace is None:
            workspace = torch.full((native.dsa_mla_prefill_workspace_size(p),), 0xAB, dtype=torch.uint8, device="cuda")
        native.dsa_mla_prefill_fwd(D["q"], D["k"], D["r"], D["v"], D["cu"], D["ck"], out, p, workspace, lse=lse)
        return out, lse, native.dsa_sparse_attn_read_status(workspace)

    def reference(self):
        d = lambda x: x.double().numpy()  # noqa: E731
        return heads.latent_attention(d(self.q), d(self.up[:, :, :128]), d(self.latent[:, 512:]), d(self.up[:, :, 128:]), self.cu, self.ck,
                                      float(np.float32(self.scale)))

    def check(self, out, lse, ref=None):
        o, l, (mass, size) = ref or self.reference()
        got, got_l = out.double().cpu().numpy(), lse.double().cpu().numpy()
        rows = ~np.isnan(l)
        assert (got[~rows] == 7.0).all() and (got_l[~rows] == 7.0).all(), "rows of no request were written"
        empty = np.isneginf(l)
        assert (got[empty] == 0).all() and np.isneginf(got_l[empty]).all()
        seen = rows & ~empty
        if not seen.any():
            return
        o, got, l, got_l, mass, size = (x[seen] for x in (o, got, l, got_l, mass, size))
        half, n = TYPES[self.dtype][1], max(b for _, b in self.lens)
        v_max = float(self.up[:, :, 128:].float().nan_to_num(0.0).abs().max())
        delta = 200 * U * size + 8 * U * (np.abs(l) + size)
        eps = (2 * (delta + 2.0 ** -21) + half + n * U)[:, None]
        bound = half * np.abs(o) + eps * mass * 1.01 + 2.0 ** -25 * (n * v_max + 1)
        bad = ~(np.abs(got - o) <= bound)
        assert not bad.any(), f"{bad.sum()} of {bad.size}, worst {np.nanmax(np.abs(got - o) / bound)} of the bound"
        bl = delta + 2.0 ** -21 + (n + 8) * U + 2 * U * np.abs(l)
        badl = ~(np.abs(got_l - l) <= bl)
        assert not badl.any(), f"lse: {badl.sum()} of {badl.size}, worst {np.nanmax(np.abs(got_l - l) / bl)} of the bound"


def _check(c, **kw):
    out, lse, status = c.run(**kw)
    assert status == 0
    c.check(out, lse)
    return out, lse


SPLIT = {"max_kv_len": 1 << 20}                                # units may be split
WHOLE = {"max_kv_len": 0}                                      # none is


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("how", [SPLIT, WHOLE], ids=["split", "whole"])
@pytest.mark.parametrize("lens", [
    [(1, 1)], [(128, 128)], [(129, 129)], [(256, 256)], [(257, 400)], [(1, 700)], [(100, 1500)], [(300, 1000)], [(5, 3), (2, 0), (0, 9), (0, 0)],
    [(130, 100), (1, 1), (64, 64), (3, 390), (255, 255)], [(33, 40)] * 9], ids=str)
def test_lengths(lens, how, dtype):
    _check(Case(len(lens), lens, dtype=dtype), **how)


def test_many_units_of_both_kinds():
    # more units than CTAs, tiles of one and two halves, several rounds
    rng = np.random.default_rng(3)
    lens = [(int(a), int(a + b)) for a, b in zip(rng.integers(0, 330, 40), rng.integers(0, 300, 40))]
    _check(Case(4, lens, h=8), **WHOLE)
    _check(Case(4, lens[:12], h=3, dtype="fp16"), **SPLIT)


def test_long_contexts_in_many_pieces():
    _check(Case(5, [(64, 20000)], h=1), **SPLIT)
    _check(Case(6, [(3, 9000), (270, 6000), (1, 50)], h=2, dtype="fp16"), **SPLIT)
    _check(Case(7, [(2, 5000)], h=16), **SPLIT)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_scores_far_apart(dtype):
    # maxima that move late, scores far below zero, and a scale of either sign and of zero
    c = Case(8, [(150, 900)], dtype=dtype, q_mag=12.0)
    c.up[3:500, :, :128] *= 0.01
    c.up[800:, :, :128] *= 6.0
    _check(c, **WHOLE)
    _check(c, **SPLIT)
    for scale in (-0.2, 0.0, 2.0):
        _check(Case(9, [(40, 300), (140, 140)], dtype=dtype, scale=scale))
    c = Case(10, [(20, 300)], dtype=dtype)
    c.latent[:, 512:] = -100.0
    c.q[:, :, 128:] = 100.0      # every score near -46000
    _check(c)
    _check(c, **SPLIT)


def test_a_query_that_is_not_finite_spoils_its_row_only():
    for how in (SPLIT, WHOLE):
        c = Case(11, [(140, 600), (3, 2)])
        want, want_l = _check(c, **how)
        c.q[5, 1, 7], c.q[90, 0, 150] = float("nan"), float("inf")
        c.q[141, 0, 3] = float("nan")    # the first row of the second request, which sees nothing
        out, lse, status = c.run(**how)
        assert status == 0 and out[5, 1].isnan().all() and lse[5, 1].isnan() and not torch.isfinite(lse[90, 0])
        assert (out[141] == 0).all() and (lse[141] == -float("inf")).all()
        keep = torch.ones_like(want_l, dtype=torch.bool)
        keep[5, 1] = keep[90, 0] = False
        assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], want_l[keep])


def test_layouts_and_no_lse():
    c = Case(12, [(77, 200), (130, 333)], h=4)
    want, want_l = _check(c)
    D = c.device()
    # heads outermost, and an output inside a wider buffer
    E = dict(D, q=D["q"].transpose(0, 1).contiguous().transpose(0, 1), k=D["k"].transpose(0, 1).contiguous().transpose(0, 1),
             v=D["v"].contiguous(), r=D["r"].contiguous())
    wide = torch.full((c.n, 6, 136), 7.0, dtype=torch.bfloat16, device="cuda")
    p = c.params(E)
    ws = torch.empty(native.dsa_mla_prefill_workspace_size(p), dtype=torch.uint8, device="cuda")
    native.dsa_mla_prefill_fwd(E["q"], E["k"], E["r"], E["v"], E["cu"], E["ck"], wide[:, 1:5, :128], p, ws)
    assert native.dsa_sparse_attn_read_status(ws) == 0
    assert torch.equal(wide[:, 1:5, :128], want)
    wide[:, 1:5, :128] = 7.0
    assert (wide == 7.0).all()


def test_empty_batches():
    z = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for n, m, cu, ck in ((0, 0, i(0), i(0)), (0, 5, i(0, 0), i(0, 5)), (4, 0, i(0, 3), i(0, 0)), (4, 0, i(0), i(0))):
        q, k, out = z(n, 2, 192), z(m, 2, 128), torch.full((n, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((n, 2), 7.0, device="cuda")
        p = native.dsa_mla_params_init(q, k, cu)
        ws = torch.full((native.dsa_mla_prefill_workspace_size(p),), 0xAB, dtype=torch.uint8, device="cuda")
        native.dsa_mla_prefill_fwd(q, k, z(m, 64), k, cu, ck, out, p, ws, lse=lse)
        assert native.dsa_sparse_attn_read_status(ws) == 0
        rows = 3 if n and cu.numel() > 1 else 0
        assert (out[:rows] == 0).all() and (out[rows:] == 7).all() and (lse[:rows] == -float("inf")).all()


def test_lengths_outside_their_range_are_taken_as_the_nearest_bound():
    c = Case(13, [(40, 90), (30, 60)])
    D = c.device()
    D["cu"], D["ck"] = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([-5, 41, c.n + 9], [-1, 93, c.m + 100]))
    D = {k: x.nan_to_num(0.0) if x.is_floating_point() else x for k, x in D.items()}
    out, lse, status = c.run(D)
    c.cu, c.ck = np.array([0, 41, c.n]), np.array([0, 93, c.m])
    c.q, c.up, c.latent = (x.nan_to_num(0.0) for x in (c.q, c.up, c.latent))
    assert status == 0
    c.check(out, lse)


def test_the_hints_change_no_result_beyond_rounding_and_calls_repeat():
    c = Case(14, [(300, 2000), (10, 700)], h=3)
    a, al, _ = c.run(max_q_len=1, max_kv_len=1)
    b, bl, _ = c.run(max_q_len=1 << 20, max_kv_len=1 << 20)
    ref = c.reference()
    c.check(a, al, ref)
    c.check(b, bl, ref)
    for kw, want, want_l in ((SPLIT, b, bl), (WHOLE, a, al)):
        for _ in range(3):
            o, l, _ = c.run(**kw)
            assert torch.equal(o, want) and torch.equal(l, want_l)


@pytest.mark.parametrize("how", [SPLIT, WHOLE], ids=["split", "whole"])
def test_captured_as_a_first_call_and_replayed_on_another_batch(how):
    c = Case(15, [(200, 500), (60, 60)], h=2)
    D = c.device()
    p = c.params(D, **how)
    ws = torch.full((native.dsa_mla_prefill_workspace_size(p),), 0xCD, dtype=torch.uint8, device="cuda")
    out = torch.full((c.n, c.h, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.n, c.h), 7.0, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            native.dsa_mla_prefill_fwd(D["q"], D["k"], D["r"], D["v"], D["cu"], D["ck"], out, p, ws, lse=lse)
    torch.cuda.synchronize()
    assert (out == 7.0).all()
    g.replay()
    torch.cuda.synchronize()
    c.check(out, lse)
    c.cu, c.ck = np.array([1, 11, c.n - 2], np.int32), np.array([3, 203, c.m - 2], np.int32)
    c.lens = [(10, 200), (c.n - 13, c.m - 205)]
    D["cu"].copy_(torch.from_numpy(c.cu))
    D["ck"].copy_(torch.from_numpy(c.ck))
    out.fill_(7.0)
    lse.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    c.check(out, lse)


def test_two_streams_with_workspaces_of_their_own():
    cs = [Case(16, [(300, 900)], h=4), Case(17, [(64, 64)] * 20, h=2, dtype="fp16")]
    Ds = [c.device() for c in cs]
    torch.cuda.synchronize()
    got = []
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(5):
        for c, D, s in zip(cs, Ds, streams):
            with torch.cuda.stream(s):
                p = c.params(D)
                ws = torch.empty(native.dsa_mla_prefill_workspace_size(p), dtype=torch.uint8, device="cuda")
                out = torch.full((c.n, c.h, 128), 7.0, dtype=TYPES[c.dtype][0], device="cuda")
                lse = torch.full((c.n, c.h), 7.0, device="cuda")
                native.dsa_mla_prefill_fwd(D["q"], D["k"], D["r"], D["v"], D["cu"], D["ck"], out, p, ws, lse=lse)
                got.append((c, out, lse, ws))
    torch.cuda.synchronize()
    refs = [c.reference() for c in cs]
    for c, out, lse, _ in got:
        c.check(out, lse, refs[cs.index(c)])


def test_offsets_past_32_bits():
    # 24k keys of 64 heads, [keys, values] side by side in rows of 400 kB: 9.6 GB
    n, h = 24000, 64
    up = torch.empty((n, h, 3136), dtype=torch.bfloat16, device="cuda")
    k, v = up[:, :, :128], up[:, :, 3008:]
    g = torch.Generator(device="cuda").manual_seed(1)
    k.copy_(torch.randn((n, h, 128), generator=g, device="cuda"))
    v.copy_(torch.randn((n, h, 128), generator=g, device="cuda"))
    assert n * h * 3136 > 2 ** 32
    r = torch.randn((n, 64), generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randn((2, h, 192), generator=g, device="cuda").to(torch.bfloat16)
    out, lse = torch.empty((2, h, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((2, h), device="cuda")
    cu, ck = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 2], [n - 300, n]))
    p = native.dsa_mla_params_init(q, k, cu)
    ws = torch.empty(native.dsa_mla_prefill_workspace_size(p), dtype=torch.uint8, device="cuda")
    native.dsa_mla_prefill_fwd(q, k, r, v, cu, ck, out, p, ws, lse=lse)
    assert native.dsa_sparse_attn_read_status(ws) == 0
    c = Case(1, [(2, 300)], h=h, pad=0)
    c.n, c.m, c.cu, c.ck = 2, 300, np.array([0, 2]), np.array([0, 300])
    c.q, c.latent = q.cpu(), torch.cat([torch.zeros((300, 512), dtype=torch.bfloat16), r[-300:].cpu()], dim=1)
    c.up = torch.cat([k[-300:], v[-300:]], dim=2).cpu()
    c.check(out, lse)


@pytest.mark.parametrize("how,lens,h", [(WHOLE, [(300, 900)] * 8, 30), (SPLIT, [(200, 9000)], 4)], ids=["whole", "split"])
def test_a_wait_that_runs_out_is_reported_and_recovered_from(how, lens, h):
    c = Case(18, lens, h=h)
    D = c.device()
    want, want_l, status = c.run(D, **how)
    assert status == 0
    t0 = time.perf_counter()
    out, lse, status = c.run(D, flags=native.DSA_MLA_FLAG_TEST_WAIT_TIMEOUT, **how)
    assert status == native.DSA_STATUS_WAIT_TIMEOUT and 0.3 < time.perf_counter() - t0 < 20.0
    same = (out == want).all(dim=-1) & (lse == want_l)
    # CTA 0's units: of 480 for 152 CTAs at most four tiles of 256 rows and heads; or its share, of two units at most
    assert int((~same).sum()) <= (4 if how is WHOLE else 2) * 256
    out, lse, status = c.run(D, **how)
    assert status == 0 and torch.equal(out, want) and torch.equal(lse, want_l)
