"""The attention over the paged 8-bit cache for requests that share prefixes (include/dsa_kv8_prefix.h) against the oracle of the
plain one (oracle/paged.py), which knows of no groups.  The error bound is that of test_kv8_attn_gpu.py with the join of two parts:
a factor 2^(m - top), exact, two products and two sums, of the result and of the softmax's sum: 8 u of mass and of lse more, within
its n u for the sums over n >= 8 cached tokens, and added here as n + 16."""

import numpy as np
import pytest
import torch

from oracle import paged
from test_kv8_attn_gpu import TYPES, Case
from top_sparse_mla_gb300 import native

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from top_sparse_mla_gb300.build import build
    build()
    native.library()


class PrefixCase(Case):
    """groups: (requests, prefix length) of each group in turn, requests of no group with prefix None.  Requests of a group share
    the pages of the whole pages of their prefix, as far as any of them reaches.  What no query sees is poisoned."""

    def __init__(self, seed, lens, groups, page=16, **kw):
        super().__init__(seed, lens, page=page, poison=False, **kw)
        rng = np.random.default_rng(seed + 1)
        at, self.cu_groups, self.prefix = 0, [0], []
        assert sum(n for n, _ in groups) == len(lens)
        for n, prefix in groups:
            if prefix is not None:
                # groups are next to each other: requests of none lie in front of the first or behind the last
                if not self.prefix:
                    self.cu_groups = [at]
                self.cu_groups.append(at + n)
                self.prefix.append(prefix)
                members = range(at, at + n)
                longest = max(members, key=lambda r: lens[r][1])
                for r in members:
                    pages = min(prefix, lens[r][1]) // page
                    self.table[r, :pages] = self.table[longest, :pages]
            at += n
        n_pages = len(self.kp)
        live = np.zeros((n_pages, page), bool)
        for r, (ql, kv) in enumerate(lens):
            used = -(-kv // page)
            self.table[r, used:] = rng.choice([-1, -5, n_pages, 2 ** 31 - 1], self.table.shape[1] - used)
            if ql:
                j = np.arange(kv)
                live[self.table[r, j // page], j % page] = True
        for p in (self.kp, self.vp):
            p[np.broadcast_to(~live[:, None, :, None], p.shape)] = 0x7F
        for s in (self.ks, self.vs):
            s[~live.any(axis=1)] = np.nan

    def device(self):
        D = super().device()
        D["cug"] = torch.tensor(self.cu_groups, dtype=torch.int32, device="cuda")
        D["pre"] = torch.tensor(self.prefix, dtype=torch.int32, device="cuda")
        return D

    def run(self, D=None, max_q_len=None, flags=0, workspace=None):
        D = D or self.device()
        out = torch.full((self.n, self.h * self.g, self.d), 7.0, dtype=TYPES[self.dtype][0], device="cuda")
        lse = torch.full((self.n, self.h * self.g), 7.0, device="cuda")
        most = max([ql for ql, _ in self.lens] + [0]) if max_q_len is None else max_q_len
        p = native.dsa_kv8_params_init(D["q"], D["kp"], D["table"], max_q_len=most, softmax_scale=self.scale, flags=flags)
        if workspace is None:
            workspace = torch.full((native.dsa_kv8_prefix_workspace_size(p, len(D["pre"])),), 0xAB, dtype=torch.uint8, device="cuda")
        native.dsa_kv8_prefix_attn_fwd(D["q"], D["kp"], D["vp"], D["ks"], D["vs"], D["table"], D["cu"], D["kv"], D["cug"], D["pre"], out,
                                       p, workspace, lse=lse)
        return out, lse, native.dsa_sparse_attn_read_status(workspace)

    def check(self, out, lse, ref=None):
        kv = self.kv
        self.kv = kv + 16   # the bound's n
        try:
            # value scales outside [2^-64, 2^64] count as the nearer bound
            vs = np.clip(self.vs, np.float32(2.0 ** -64), np.float32(2.0 ** 64))
            super().check(out, lse, ref or paged.kv8_attention(self.q.double().numpy(), self.kp, self.vp, self.ks, vs, self.table,
                                                               self.cu, kv, float(np.float32(self.scale)), 0))
        finally:
            self.kv = kv


def _check(c, **kw):
    out, lse, status = c.run(**kw)
    assert status == 0
    c.check(out, lse)
    return out, lse


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 16), (128, 64), (64, 128), (128, 32)])
@pytest.mark.parametrize("lens,groups", [
    ([(1, 300)] * 4, [(4, 256)]),                                             # few rows
    ([(1, 200 + 7 * i) for i in range(40)], [(40, 190)]),                     # more than one tile
    ([(1, 90), (1, 500), (1, 300), (2, 301), (1, 299), (1, 700), (1, 701)], [(2, None), (3, 290), (1, 600), (1, None)]),
    ([(1, 1), (1, 64), (1, 65), (1, 200)], [(4, 64)]),                        # a request that does not reach the prefix's end
    ([(0, 300), (1, 300), (0, 0), (3, 260), (5, 261)], [(5, 256)]),           # without queries, and drafted tokens
    ([(40, 440), (1, 401), (60, 460), (300, 700)], [(4, 400)]),               # chunks of prompts behind a shared prompt
    ([(20, 20), (30, 30)], [(2, 16)]),                                        # queries inside the prefix: nothing is shared
    ([(1, 2000), (1, 1990), (4, 1999)] * 3, [(3, 1984), (3, 64), (3, 1024)]),
], ids=["few", "tiles", "some of none", "short of it", "no queries", "chunks", "inside", "three groups"])
def test_groups(lens, groups, d, page, dtype):
    for h, g in ((2, 4), (1, 8)):
        _check(PrefixCase(d + page, lens, groups, page=page, h=h, g=g, d=d, dtype=dtype))


@pytest.mark.parametrize("g", [1, 3, 16, 40, 128])
def test_group_sizes(g):
    lens = [(1, 400 + i) for i in range(7)]
    _check(PrefixCase(g, lens, [(7, 390)], h=2 if g < 40 else 1, g=g, d=64))
    _check(PrefixCase(g, lens, [(7, 390)], h=3 if g < 40 else 1, g=g, d=128, dtype="fp16"))


def test_large_groups_and_long_prefixes():
    _check(PrefixCase(3, [(1, 6000 + 3 * i) for i in range(40)], [(40, 5999)], page=64, h=1, g=8))
    _check(PrefixCase(4, [(2, 1500 + i) for i in range(200)], [(70, 1490), (130, 1490)], page=128, h=2, g=2, d=64, dtype="fp16"))


@pytest.mark.parametrize("d", [64, 128])
def test_many_requests(d):
    # more parts than the plan's threads
    rng = np.random.default_rng(5)
    lens = [(1, int(x)) for x in rng.integers(40, 90, 1500)]
    _check(PrefixCase(6, lens, [(500, 32), (3, 40), (997, 48)], page=16, h=1, g=2, d=d))


@pytest.mark.parametrize("n,groups", [(4096, [(1, 16)] * 4096), (8191, [(8191, 16)]), (6000, [(3, 16)] * 2000)])
def test_as_many_requests_and_groups_as_there_may_be(n, groups):
    assert n + len(groups) <= native.DSA_KV8_MAX_REQ and len(groups) <= native.DSA_KV8_MAX_GROUPS
    _check(PrefixCase(21, [(1, 18 + i % 3) for i in range(n)], groups, page=16, h=1, g=2, d=64))


def test_without_groups_and_with_groups_of_one():
    lens = [(1, 300), (9, 70), (1, 1), (0, 0), (2, 513)]
    c = PrefixCase(7, lens, [(5, None)], h=2, g=4)
    c.cu_groups = [0]
    _check(c)
    _check(PrefixCase(7, lens, [(1, 256), (1, 64), (1, 16), (1, 0), (1, -3)], h=2, g=4))


def test_less_than_is_shared_and_more_than_is_seen():
    c = PrefixCase(8, [(1, 300 + i) for i in range(9)], [(9, 288)])
    want, want_l = _check(c)
    for prefix in (0, 15, 16, 100):
        c.prefix = [prefix]
        _check(c)
    # pages behind what a request sees are not looked at: the group shares what all of it sees
    c = PrefixCase(9, [(1, 300), (3, 100), (1, 290)], [(3, 288)])
    c.prefix = [1 << 30]
    c.table[0, 6:], c.table[2, 6:] = c.table[0, 6:].copy(), c.table[2, 6:].copy()
    _check(c)


def test_lists_of_groups_outside_their_range():
    c = PrefixCase(10, [(1, 200), (1, 210), (2, 220)], [(3, 192)])
    c.cu_groups = [-7, 99]
    _check(c)


def test_scales_far_apart_and_scores_far_apart():
    for d in (64, 128):
        for scales in ([2.0 ** -60, 2.0 ** 60], [2.0 ** -40, 1.0], [2.0 ** -140, 2.0 ** 120]):
            _check(PrefixCase(11, [(1, 300 + i) for i in range(20)], [(20, 290)], d=d, v_scale=scales))
            _check(PrefixCase(12, [(1, 300 + i) for i in range(2)], [(2, 290)], d=d, v_scale=scales))
        _check(PrefixCase(13, [(1, 300 + i) for i in range(20)], [(20, 290)], d=d, k_mag=20.0))
        _check(PrefixCase(14, [(1, 300 + i) for i in range(20)], [(20, 290)], d=d, scale=-0.3, dtype="fp16"))


def test_a_query_that_is_not_finite_spoils_its_rows_only():
    c = PrefixCase(15, [(1, 200 + i) for i in range(40)], [(40, 192)], h=1, g=8)
    want, want_l = _check(c)
    clean = c.q[3, 2, 5].clone(), c.q[30, 7, 0].clone()
    c.q[3, 2, 5], c.q[30, 7, 0] = float("nan"), float("inf")
    out, lse, status = c.run()
    assert status == 0 and out[3, 2].isnan().all() and lse[3, 2].isnan()
    # Other rows need not be the same bits: a warp sets the running maxima of its 8 rows anew when one of them asks for it, and each
    # product of a row's sum with the factor is rounded by u (its O's the same), once for a step of 16 tokens at most.  That is
    # within the bound, whose n u has u for every token; the rows in question are those of the clean call there.
    for t, h in ((3, 2), (30, 7)):
        out[t, h], lse[t, h] = want[t, h], want_l[t, h]
    c.q[3, 2, 5], c.q[30, 7, 0] = clean
    c.check(out, lse)


def test_a_request_with_too_many_queries_is_skipped():
    lens = [(1, 300), (4, 310), (1, 320)]
    c = PrefixCase(16, lens, [(3, 256)], h=2, g=4)
    out, lse, status = c.run(max_q_len=3)
    assert status == native.DSA_STATUS_QUERY_TOO_LONG
    ref = list(paged.kv8_attention(c.q.double().numpy(), c.kp, c.vp, c.ks, c.vs, c.table, c.cu, c.kv, float(np.float32(c.scale)), 0))
    ref[0][2:6], ref[1][2:6] = np.nan, np.nan
    c.check(out, lse, tuple(ref))


def test_pages_that_do_not_exist_are_not_seen():
    for n in (2, 30):
        c = PrefixCase(17, [(1, 400)] * n, [(n, 384)], h=1, g=8, page=16)
        for r in range(n):
            c.table[r, 3], c.table[r, 10] = -1, len(c.kp) + 5
        c.table[1, 24] = -2
        _check(c)
        c.table[:, :] = -1
        out, lse, status = c.run()
        assert status == 0 and (out[1:n + 1] == 0).all() and (lse[1:n + 1] == -float("inf")).all()


def test_the_same_inputs_give_the_same_bits_as_often_as_asked():
    c = PrefixCase(18, [(1, 2100 + 31 * i) for i in range(24)], [(24, 2048)], h=2, g=8, d=128, page=64)
    D = c.device()
    want, want_l = _check(c)
    for _ in range(5):
        out, lse, _ = c.run(D)
        assert torch.equal(out, want) and torch.equal(lse, want_l)


@pytest.mark.parametrize("n", [3, 40])
def test_captured_as_a_first_call_and_replayed_on_another_batch(n):
    c = PrefixCase(19, [(1, 300 + i) for i in range(n)], [(n, 288)], h=2, g=8)
    D = c.device()
    p = native.dsa_kv8_params_init(D["q"], D["kp"], D["table"], max_q_len=1)
    ws = torch.full((native.dsa_kv8_prefix_workspace_size(p, 1),), 0xCD, dtype=torch.uint8, device="cuda")
    out = torch.full((c.n, 16, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.n, 16), 7.0, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            native.dsa_kv8_prefix_attn_fwd(D["q"], D["kp"], D["vp"], D["ks"], D["vs"], D["table"], D["cu"], D["kv"], D["cug"], D["pre"],
                                           out, p, ws, lse=lse)
    torch.cuda.synchronize()
    assert (out == 7.0).all()
    for shorter in (0, 1, 40, 0):
        c.kv = np.array([300 + i - shorter for i in range(n)], np.int32)
        c.lens = [(1, int(x)) for x in c.kv]
        c.prefix = [288 if shorter < 40 else 64]
        D["kv"].copy_(torch.from_numpy(c.kv))
        D["pre"].copy_(torch.tensor(c.prefix))
        out.fill_(7.0)
        lse.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        c.check(out, lse)


def test_a_wait_that_runs_out_is_reported_and_recovered_from():
    c = PrefixCase(20, [(1, 4000 + i) for i in range(300)], [(300, 3990)], page=128, h=2, g=8, d=64)
    D = c.device()
    want, want_l, status = c.run(D)
    assert status == 0
    _, _, status = c.run(D, flags=native.DSA_KV8_FLAG_TEST_WAIT_TIMEOUT)
    assert status == native.DSA_STATUS_WAIT_TIMEOUT
    out, lse, status = c.run(D)
    assert status == 0 and torch.equal(out, want) and torch.equal(lse, want_l)
