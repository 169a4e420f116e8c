"""The attention over the paged 8-bit cache (include/dsa_kv8.h) against the oracle
(oracle/paged.py) in float64.

Error bound of an output value o = sum_j p_j v_j (derived from the stated numerics, before
any run), with u = 2^-24:
  - rounding of the result: half a step, 2^-8 |o| (bf16) or 2^-11 |o| (fp16), and half of
    the smallest fp16 step, 2^-25, where it is subnormal;
  - each score has an error of at most delta: q and the codes are exact but for q values
    below 2^-30 of their row's largest (in all 2^-30 d of the largest product, below the
    next term); the sum of d products in fp32 in any order, then four more roundings, and
    the maximum's own size in the exponent: delta <= (d + 8) u size + 8 u (|lse| + size + 64)
    with size = max_j sum_i |q_i k_ij| * softmax_scale (the 64 is the largest |log2
    v_scale|); the exponential adds 2^-21 relative.  A relative error eps of every weight
    changes o by at most 2 eps sum_j p_j |v_j|;
  - the weights' rounding to fp16: 2^-11 relative of each normal one, half the smallest
    step 2^-25 of the subnormal ones, against a largest weight of at least 1:
    2^-11 mass + 2^-25 tiny, tiny = max_j(p_j v_scale_j) sum_j |code_j|;
  - the fp32 sums over the n cached tokens: n u mass.
lse: delta + 2^-21 + (n + 8) u."""

import numpy as np
import pytest
import torch

from oracle import codecs, paged
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
    """lens: (q_len, kv_len) of each request.  Everything that no query sees is poisoned: NaN codes and scales, pages
    that do not exist."""

    def __init__(self, seed, lens, h=2, g=4, d=128, page=64, dtype="bf16", window=0, k_mag=1.0, v_scale=None, q_mag=2.0,
                 pad=2, cols_more=1, poison=True, scale=None):
        rng = np.random.default_rng(seed)
        self.h, self.g, self.d, self.page, self.dtype, self.window = h, g, d, page, dtype, window
        self.scale = d ** -0.5 if scale is None else scale
        self.lens = lens
        n = len(lens)
        pages = [-(-kv // page) for _, kv in lens]
        cols = max(pages + [0]) + cols_more
        n_pages = sum(pages) + 3
        order = rng.permutation(n_pages)
        self.table = np.full((n, cols), -1, np.int32)
        if poison:
            self.table[:, :] = rng.choice([-1, -5, n_pages, 2 ** 31 - 1], self.table.shape)
        at = 0
        for r, p in enumerate(pages):
            self.table[r, :p] = order[at:at + p]
            at += p

        def pool():
            x = rng.standard_normal((n_pages, h, page, d)) * 60.0
            return codecs.e4m3_encode(x)

        self.kp, self.vp = pool(), pool()
        self.ks = (k_mag / 60.0 * np.exp2(rng.uniform(-1, 1, (n_pages, h)))).astype(np.float32)
        self.vs = (1.0 / 60.0 * np.exp2(rng.uniform(-2, 2, (n_pages, h)))).astype(np.float32)
        if v_scale is not None:
            self.vs = rng.choice(np.asarray(v_scale, np.float32), (n_pages, h))
        if poison:
            live = np.zeros((n_pages, page), bool)
            for r, (ql, kv) in enumerate(lens):
                if ql == 0:
                    continue
                lo = max(kv - ql - window + 1, 0) if window else 0
                for j in range(lo, kv):
                    live[self.table[r, j // page], j % page] = True
            for p in (self.kp, self.vp):
                p[np.broadcast_to(~live[:, None, :, None], p.shape)] = 0x7F
            for s in (self.ks, self.vs):
                s[~live.any(axis=1)] = np.nan
        self.cu = np.concatenate([[1], 1 + np.cumsum([ql for ql, _ in lens])]).astype(np.int32)   # row 0 belongs to nobody
        self.kv = np.array([kv for _, kv in lens], np.int32)
        self.n = int(self.cu[-1]) + pad
        q = torch.from_numpy(rng.standard_normal((self.n, h * g, d)) * q_mag).to(TYPES[dtype][0])
        self.q = q
        q[0] = float("nan")
        q[self.n - pad:] = float("nan")

    def device(self):
        t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        return {"q": self.q.cuda(), "kp": t(self.kp), "vp": t(self.vp), "ks": t(self.ks), "vs": t(self.vs), "table": t(self.table),
                "cu": t(self.cu), "kv": t(self.kv)}

    def run(self, dev=None, out=None, max_q_len=None, stream=None, workspace=None, lse=True):
        D = dev or self.device()
        if out is None:
            out = torch.full((self.n, self.h * self.g, self.d), 7.0, dtype=TYPES[self.dtype][0], device="cuda")
        ls = torch.full((self.n, self.h * self.g), 7.0, device="cuda") if lse else None
        most = max([ql for ql, _ in self.lens] + [0]) if max_q_len is None else max_q_len
        p = native.dsa_kv8_params_init(D["q"], D["kp"], D["table"], max_q_len=most, window=self.window, softmax_scale=self.scale)
        if workspace is None:
            workspace = torch.full((native.dsa_kv8_attn_workspace_size(p),), 0xAB, dtype=torch.uint8, device="cuda")
        native.dsa_kv8_attn_fwd(D["q"], D["kp"], D["vp"], D["ks"], D["vs"], D["table"], D["cu"], D["kv"], out, p, workspace,
                                lse=ls, stream=stream)
        status = native.dsa_sparse_attn_read_status(workspace)
        return out, ls, status

    def reference(self):
        return paged.kv8_attention(self.q.double().numpy(), self.kp, self.vp, self.ks, self.vs, self.table, self.cu, self.kv,
                                   float(np.float32(self.scale)), self.window)

    def check(self, out, lse, ref=None):
        o, l, (mass, tiny, size) = self.reference() if ref is None else ref
        got, got_l = out.double().cpu().numpy(), lse.double().cpu().numpy()
        rows = ~np.isnan(l)
        assert (got[~rows] == 7.0).all() and (got_l[~rows] == 7.0).all(), "rows of no request were written"
        empty = np.isneginf(l)
        assert (got[empty] == 0).all() and np.isneginf(got_l[empty]).all()
        seen = rows & ~empty
        if not seen.any():
            return
        o, got, l, got_l, mass, tiny, size = (x[seen] for x in (o, got, l, got_l, mass, tiny, size))
        n = max(self.kv.max(), 1)
        delta = (self.d + 8) * U * size + 8 * U * (np.abs(l) + size + 64)
        eps = (2 * (delta + 2.0 ** -21) + 2.0 ** -11 + n * U)[:, None]
        bound = TYPES[self.dtype][1] * np.abs(o) + eps * mass * 1.01 + 2.0 ** -25 * (tiny + 1)
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


DECODE = [(1, 1), (1, 15), (1, 16), (1, 17), (1, 0), (0, 40), (1, 64), (1, 129), (1, 1000), (0, 0), (1, 333)]


@pytest.mark.parametrize("d,page,dtype,h,g", [
    (128, 64, "bf16", 2, 8), (128, 16, "fp16", 3, 4), (128, 128, "bf16", 1, 1), (64, 32, "fp16", 2, 8), (64, 16, "bf16", 1, 5),
    (128, 32, "fp16", 2, 12), (64, 64, "bf16", 2, 16), (128, 64, "bf16", 1, 24), (64, 128, "fp16", 1, 32), (128, 16, "bf16", 1, 40),
    (64, 16, "fp16", 1, 128)])
@pytest.mark.parametrize("window", [0, 1, 100])
def test_single_queries(d, page, dtype, h, g, window):
    _check(Case(d + g + window, DECODE, h=h, g=g, d=d, page=page, dtype=dtype, window=window))


VERIFY = [(3, 3), (2, 40), (4, 17), (1, 70), (0, 9), (4, 257), (3, 2), (4, 0), (2, 64)]


@pytest.mark.parametrize("d,page,dtype,h,g", [(128, 32, "bf16", 2, 4), (64, 16, "fp16", 2, 8), (128, 64, "fp16", 1, 2),
                                              (128, 16, "bf16", 2, 1), (64, 128, "bf16", 1, 8)])
@pytest.mark.parametrize("window", [0, 2, 33])
def test_a_few_queries_per_request(d, page, dtype, h, g, window):
    # (3, 2) and (4, 0): queries before the sequence's start see nothing
    _check(Case(d + g + window, VERIFY, h=h, g=g, d=d, page=page, dtype=dtype, window=window))


PREFILL = [(130, 130), (1, 77), (65, 300), (0, 5), (40, 39), (17, 17), (129, 515)]


@pytest.mark.parametrize("d,page,dtype,h,g", [(128, 64, "bf16", 2, 4), (128, 16, "fp16", 1, 8), (64, 32, "bf16", 2, 3),
                                              (64, 128, "fp16", 1, 1), (128, 128, "bf16", 1, 5)])
@pytest.mark.parametrize("window", [0, 1, 50, 200])
def test_prefill_and_mixed_batches(d, page, dtype, h, g, window):
    _check(Case(d + g + window, PREFILL, h=h, g=g, d=d, page=page, dtype=dtype, window=window))


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 30, 5000])
def test_windows_wider_than_every_context(window):
    # (3, 2) and (70, 60): queries at negative positions, whose window would begin before -2^31
    for lens in ([(1, 40), (3, 2), (2, 90)], [(70, 60), (130, 400)]):
        c, e = Case(32, lens, h=1, g=4, page=16, window=window), Case(32, lens, h=1, g=4, page=16)
        a, b = _check(c), _check(e)
        assert torch.equal(a[0][1:-2], b[0][1:-2]) and torch.equal(a[1], b[1])


def test_groups_of_many_heads_in_prefill():
    _check(Case(3, [(9, 30), (33, 100)], h=1, g=16, page=16))
    _check(Case(4, [(3, 30), (5, 100)], h=1, g=128, d=64, page=32, dtype="fp16"))
    _check(Case(5, [(7, 200), (2, 11)], h=2, g=33, page=64))


def test_long_contexts_split_over_many_ctas():
    _check(Case(6, [(1, 20000)], h=1, g=8, page=64))
    _check(Case(7, [(1, 9000), (1, 3), (4, 12001), (1, 640)], h=2, g=2, page=32, dtype="fp16"))
    _check(Case(8, [(1, 9000), (2, 7000)], h=1, g=16, d=64, page=128, window=3000))
    _check(Case(9, [(150, 5000), (1, 9000)], h=1, g=2, page=16))


def test_many_requests():
    rng = np.random.default_rng(10)
    _check(Case(11, [(1, int(x)) for x in rng.integers(0, 60, 1500)], h=1, g=2, d=64, page=16))
    _check(Case(12, [(int(a), int(b)) for a, b in zip(rng.integers(0, 6, 300), rng.integers(0, 40, 300))], h=2, g=4, d=64, page=16,
                dtype="fp16"))


@pytest.mark.parametrize("n", [127, 128, 129, 513, 1536, 1537])
@pytest.mark.parametrize("kw", [dict(h=1, g=2, d=128), dict(h=3, g=12, d=64)])
def test_batches_at_the_sizes_where_the_shares_are_found_otherwise(n, kw):
    rng = np.random.default_rng(n)
    _check(Case(n, [(int(a), int(b)) for a, b in zip(rng.integers(0, 3, n), rng.integers(0, 50, n))], page=16, **kw))


@pytest.mark.parametrize("lens,h,g", [
    ([(1, 30000)], 1, 4),                       # all CTAs on one unit, joined in two levels
    ([(1, 6000), (0, 10), (1, 5), (1, 2500)], 2, 8),
    ([(2, 9000), (1, 700)], 3, 8),
    ([(4, 5000), (3, 5001)], 4, 8),
    ([(1, 300 + 7 * i) for i in range(38)], 2, 2),   # two CTAs a unit, on 152
    ([(1, 300 + 7 * i) for i in range(39)], 2, 2),
    ([(1, 4000)] + [(1, 1 + 17 * i) for i in range(37)], 2, 2),
    ([(1, 1 + 17 * i) for i in range(38)] + [(1, 4000)], 2, 2),
])
def test_few_units_shared_by_wide_ctas(lens, h, g):
    _check(Case(40, lens, h=h, g=g, page=64))
    _check(Case(41, lens, h=h, g=g, page=16, window=900, dtype="fp16"))
    _check(Case(42, lens, h=h, g=g, page=32, window=3600))


# 12, 10, 8, 6, 4 and 2 CTAs for each tile and head, on 152
@pytest.mark.parametrize("h,kw", [(h, dict(d=128, page=64)) for h in (1, 5, 7, 10, 16, 30)] +
                         [(h, kw) for h in (2, 6) for kw in (dict(d=64, page=16, dtype="fp16"), dict(d=128, page=32, window=1700))])
def test_a_few_tiles_whose_blocks_are_split_over_a_cluster(h, kw):
    _check(Case(50 + h, [(33, 3101)], h=h, g=8, **kw))


def test_split_tiles_with_halves_that_end_apart():
    _check(Case(60, [(200, 700)], h=1, g=2, page=16))               # the halves' last blocks differ
    _check(Case(61, [(17, 2000), (40, 41), (9, 9)], h=2, g=8))      # a half without rows; a tile too short to split
    _check(Case(62, [(100, 0), (90, 60), (33, 2500)], h=1, g=8))    # rows that see nothing
    _check(Case(63, [(256, 4000)], h=1, g=1, window=130, page=32))  # pieces that some rows do not see at all
    _check(Case(64, [(250, 250), (3, 4000)], h=1, g=3, d=64, page=16))


@pytest.mark.parametrize("kw", [
    dict(v_scale=[2.0 ** -64, 2.0 ** -40]), dict(v_scale=[2.0 ** 40, 2.0 ** 39]), dict(v_scale=[2.0 ** -30, 1.0, 2.0 ** 10]),
    dict(q_mag=2.0 ** 60, k_mag=2.0 ** -60), dict(q_mag=2.0 ** -60, k_mag=2.0 ** 60), dict(q_mag=30.0), dict(scale=-0.1),
    dict(scale=0.0)])
@pytest.mark.parametrize("lens", [[(1, 300), (2, 50)], [(70, 300)]])
def test_magnitudes(kw, lens):
    c = Case(13, lens, h=1, g=4, page=32, **kw)
    if "v_scale" in kw:   # the output's own type has to hold the values
        assert np.abs(c.reference()[0][1:-2]).max() < 3e38
    _check(c)


@pytest.mark.parametrize("low,high", [(8, 22), (14, 26), (14, 30), (15, 40)])
def test_scores_that_rise_within_and_between_blocks(low, high):
    """Scores 0 for 128 tokens, then 64 at 2^low times their weight, then one at 2^high: what the 64 add up to is 64 * 2^(low - high)
    of the mass, up to 1.5 %, and must not get lost when the maximum is moved."""
    c = Case(70, [(40, 256)], h=1, g=8, d=128, page=16, v_scale=[1.0], poison=False, scale=float(np.log(2.0)))
    c.ks[:] = 1.0
    c.q[:] = 0.0
    c.q[:, :, 0] = 1.0
    c.kp[:] = 0
    for j in range(128, 256):
        c.kp[c.table[0, j // 16], 0, j % 16, 0] = codecs.e4m3_encode(np.array([low if j < 192 else high if j == 200 else 0.0]))[0]
    _check(c)


def test_queries_with_a_wide_range_in_one_row_and_zero_rows():
    c = Case(14, [(1, 200), (40, 120)], h=1, g=4, page=16)
    c.q[1:-2, :, ::3] *= 2.0 ** -12
    c.q[1:-2, 0] = 0.0
    _check(c)


def test_all_pages_missing_sees_nothing():
    c = Case(15, [(1, 100), (2, 30), (50, 80)], h=1, g=2, page=16)
    c.table[:] = -1
    out, lse = _check(c)
    assert (out[1:-2] == 0).all()
    # one page missing in the middle
    c = Case(16, [(1, 100), (2, 90), (50, 80)], h=1, g=2, page=16, poison=False)
    c.table[:, 2] = 10 ** 6
    _check(c)


def test_strided_queries_outputs_and_tables():
    c = Case(17, [(1, 70), (3, 40), (50, 90)], h=2, g=2, d=64, page=16)
    D = c.device()
    wide = torch.full((c.n, c.h * c.g + 3, 2 * c.d), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 1:1 + c.h * c.g, :c.d] = D["q"]
    D["q"] = wide[:, 1:1 + c.h * c.g, :c.d]
    heads_first = torch.full((c.h * c.g, c.n, c.d), 7.0, dtype=torch.bfloat16, device="cuda")
    tab = torch.full((len(c.lens), c.table.shape[1] + 5), 3, dtype=torch.int32, device="cuda")
    tab[:, :c.table.shape[1]] = D["table"]
    D["table"] = tab[:, :c.table.shape[1]]
    out, lse, status = c.run(dev=D, out=heads_first.transpose(0, 1))
    assert status == 0
    c.check(out, lse)


def test_without_lse_the_output_is_the_same():
    c = Case(18, [(1, 500), (40, 90)], h=2, g=4)
    a, _, _ = c.run()
    b, _, _ = c.run(lse=False)
    assert torch.equal(a, b)


def test_the_same_call_gives_the_same_bits():
    for lens in ([(1, 7000), (2, 3000), (1, 5)], [(200, 700), (1, 40)]):
        c = Case(19, lens, h=2, g=8)
        D = c.device()
        a = c.run(dev=D)
        for _ in range(5):
            b = c.run(dev=D)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_a_request_with_too_many_queries_is_reported_and_skipped():
    for lens, most in (([(1, 40), (3, 50), (1, 9)], 2), ([(100, 150), (200, 300), (1, 9)], 120)):
        c = Case(20, lens, h=1, g=4, page=16)
        out, lse, status = c.run(max_q_len=most)
        assert status == native.DSA_STATUS_QUERY_TOO_LONG
        a, b = c.cu[1], c.cu[2]
        assert (out[a:b] == 7).all() and (lse[a:b] == 7).all()
        keep = np.ones(c.n, bool)
        keep[a:b] = False
        o, l, (m, t, s) = c.reference()
        l[a:b] = np.nan
        c.check(out, lse, (o, l, (m, t, s)))


def test_a_larger_bound_on_the_queries_changes_only_the_launches():
    c = Case(21, [(1, 200), (2, 90), (1, 31)], h=2, g=4, page=16)
    for most in (2, 9, 1000):
        out, lse, status = c.run(max_q_len=most)
        assert status == 0
        c.check(out, lse)


def test_empty_batches():
    c = Case(22, [], h=1, g=2, pad=3, cols_more=0)
    out, lse, status = c.run()
    assert status == 0 and (out == 7).all() and (lse == 7).all()
    c = Case(23, [(0, 5), (0, 0)], h=1, g=2, page=16, pad=3)
    out, lse, status = c.run()
    assert status == 0 and (out == 7).all()
    c = Case(24, [(2, 0), (1, 0)], h=1, g=2, page=16, cols_more=0)   # a table without columns
    _check(c)


def test_a_pool_past_32_bits():
    # 2.2 GB a pool, the request's pages at its end
    n_pages, h, page, d = 8448, 16, 128, 128
    c = Case(25, [(1, 700), (130, 300)], h=h, g=1, page=page, d=d, poison=False)
    D = c.device()
    k = c.kp.shape[0]
    for name in ("kp", "vp"):
        big = torch.full((n_pages, h, page, d), 0x7F, dtype=torch.uint8, device="cuda")
        big[-k:] = D[name]
        D[name] = big
    for name in ("ks", "vs"):
        big = torch.full((n_pages, h), float("nan"), device="cuda")
        big[-k:] = D[name]
        D[name] = big
    D["table"] = torch.where(D["table"] >= 0, D["table"] + (n_pages - k), D["table"])
    out, lse, status = c.run(dev=D)
    assert status == 0
    c.check(out, lse)


@pytest.mark.parametrize("lens", [[(1, 3000), (1, 40), (2, 500)], [(150, 400), (1, 90)]])
def test_replayed_from_graphs_that_share_a_workspace(lens):
    c, e = Case(26, lens, h=2, g=4), Case(27, list(reversed(lens)), h=2, g=4)
    ref = [x.run() for x in (c, e)]
    most = max(q for q, _ in lens)
    devs, outs, graphs, ws = [x.device() for x in (c, e)], [], [], None
    for x, D in zip((c, e), devs):
        p = native.dsa_kv8_params_init(D["q"], D["kp"], D["table"], max_q_len=most, softmax_scale=x.scale)
        if ws is None:
            ws = torch.empty(native.dsa_kv8_attn_workspace_size(p), dtype=torch.uint8, device="cuda")
        out = torch.full((x.n, x.h * x.g, x.d), 7.0, dtype=torch.bfloat16, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            native.dsa_kv8_attn_fwd(D["q"], D["kp"], D["vp"], D["ks"], D["vs"], D["table"], D["cu"], D["kv"], out, p, ws)
        outs.append(out)
        graphs.append(graph)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for out, r in zip(outs, ref):
        assert torch.equal(out, r[0])


def test_on_another_stream_and_two_calls_at_once():
    c, e = Case(28, [(1, 5000), (1, 100)], h=2, g=8), Case(29, [(90, 900)], h=2, g=4)
    ref = [x.run() for x in (c, e)]
    devs = [x.device() for x in (c, e)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    outs = [torch.full((x.n, x.h * x.g, x.d), 7.0, dtype=torch.bfloat16, device="cuda") for x in (c, e)]
    ps, wss = [], []
    for x, D in zip((c, e), devs):
        p = native.dsa_kv8_params_init(D["q"], D["kp"], D["table"], max_q_len=max(q for q, _ in x.lens), softmax_scale=x.scale)
        ps.append(p)
        wss.append(torch.empty(native.dsa_kv8_attn_workspace_size(p), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    for _ in range(4):
        for D, out, p, ws, s in zip(devs, outs, ps, wss, streams):
            native.dsa_kv8_attn_fwd(D["q"], D["kp"], D["vp"], D["ks"], D["vs"], D["table"], D["cu"], D["kv"], out, p, ws, stream=s)
    torch.cuda.synchronize()
    for out, r in zip(outs, ref):
        assert torch.equal(out, r[0])


def test_a_workspace_that_is_too_small_is_refused():
    c = Case(30, [(1, 50)], h=1, g=2)
    with pytest.raises(native.DsaError) as err:
        c.run(workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    assert err.value.code == native.DSA_ERR_WORKSPACE_TOO_SMALL


def test_tensors_that_do_not_fit_are_refused():
    c = Case(31, [(1, 50), (1, 20)], h=1, g=2)
    D = c.device()
    n = len(c.lens)
    one_row = D["table"][:1].expand(n, -1)                       # rows that overlap
    for name, bad in (("table", one_row), ("table", D["table"].long()), ("table", D["table"].t().contiguous().t()[:, :1]),
                      ("cu", D["cu"][:-1]), ("kv", D["kv"].cpu()), ("ks", D["ks"].double()), ("vs", D["vs"][:-1]),
                      ("vp", D["vp"].transpose(2, 3)), ("q", D["q"].half()), ("q", D["q"][:, :1]), ("kp", D["kp"][:, :, :8])):
        p = native.dsa_kv8_params_init(D["q"], D["kp"], D["table"], max_q_len=1)
        E = dict(D, **{name: bad})
        out = torch.full((c.n, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(native.dsa_kv8_attn_workspace_size(p), dtype=torch.uint8, device="cuda")
        if name == "table" and bad.dtype == torch.int32 and bad.shape[1] == 1 and p.table_cols == 1:
            continue
        with pytest.raises(native.DsaError) as err:
            native.dsa_kv8_attn_fwd(E["q"], E["kp"], E["vp"], E["ks"], E["vs"], E["table"], E["cu"], E["kv"], out, p, ws)
        assert err.value.code == native.DSA_ERR_INVALID_ARG
        assert (out == 7).all()
