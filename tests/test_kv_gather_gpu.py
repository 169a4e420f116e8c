"""Latent rows read back from the cache (include/dsa_kv_gather.h) against the oracle (oracle/heads.py).

A value is code * scale, rounded to fp32 (2^-24) and then to bf16 (2^-8 of the value): at most (2^-8 + 2^-24) (1 + 2^-8) of
it.  The rotary values are bits."""

import numpy as np
import pytest
import torch

from oracle import heads
from oracle.kv_insert import kv_insert
from top_sparse_mla_gb300 import native

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from top_sparse_mla_gb300.build import build
    build()
    native.library()


def _pool(n_rows, seed):
    rng = np.random.default_rng(seed)
    pool = rng.integers(0, 256, (n_rows, 656), dtype=np.uint8)
    codes = pool[:, :512]
    codes[(codes & 0x7F) == 0x7F] = 0x3A   # no NaN codes
    scale = np.exp2(rng.uniform(-12, 6, (n_rows, 4))).astype(np.float32)
    pool[:, 512:528] = scale.view(np.uint8)
    pool[:, 528:] = torch.from_numpy(rng.standard_normal((n_rows, 64)).astype(np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint8)
    return pool


def _run(pool, table, cu, page, n_out, lens=None, ld=576, status=True):
    out = torch.full((n_out, ld), 7.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda") if status else None
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    native.dsa_kv_gather(t(pool), t(table), t(np.asarray(cu, np.int32)), out, page, lens=None if lens is None else t(np.asarray(lens, np.int32)),
                         status=st)
    return out, st.item() if status else None


def _check(pool, table, cu, page, n_out, lens=None, ld=576):
    out, st = _run(pool, table, cu, page, n_out, lens, ld)
    want, missing = heads.kv_gather(pool, table, cu, lens, page, n_out)
    got = out.double().cpu().numpy()
    assert (got[:, 576:] == 7).all()
    none = np.isnan(want[:, 0])
    assert (got[none] == 7).all(), "rows of nobody were written"
    want, got = want[~none], got[~none, :576]
    assert (np.abs(got - want) <= 1.01 * 2.0 ** -8 * np.abs(want)).all()
    assert np.array_equal(got[:, 512:], want[:, 512:])
    assert st == (native.DSA_STATUS_SLOT_OUT_OF_RANGE if missing else 0)


@pytest.mark.parametrize("page", [1, 7, 16, 64, 128])
@pytest.mark.parametrize("lens,pad", [([1], 0), ([0], 2), ([33, 0, 1, 64, 127, 0], 3), ([5] * 70, 0), ([700, 3], 1)])
def test_ragged(page, lens, pad):
    rng = np.random.default_rng(page + len(lens))
    pages = [-(-n // page) for n in lens]
    order = rng.permutation(sum(pages) + 2).astype(np.int32)
    table = np.full((len(lens), max(max(pages), 1) + 1), -1, np.int32)
    at = 0
    for r, p in enumerate(pages):
        table[r, :p] = order[at:at + p]
        at += p
    cu = np.concatenate([[1], 1 + np.cumsum(lens)])   # row 0 is nobody's
    pool = _pool((sum(pages) + 2) * page, page)
    _check(pool, table, cu, page, int(cu[-1]) + pad)
    some = [rng.integers(-1, n + 3) for n in lens]
    _check(pool, table, cu, page, int(cu[-1]) + pad, lens=some, ld=592)


def test_places_that_do_not_exist_are_zero():
    pool = _pool(64, 1)
    table = np.array([[3, -1, 4, 0], [2 ** 31 - 1, 1, -2 ** 31, 2]], np.int32)
    _check(pool, table, [0, 64, 128], 16, 128)          # page 4 is past the pool
    _check(pool, table, [0, 70, 130], 16, 130)          # rows past the table's columns
    _check(pool[:60], table, [0, 64, 128], 16, 128)     # a pool that ends inside a page
    _check(pool, table, [0, 300, 20], 16, 128)          # past n_out, and back: taken as the nearest bound
    _run(pool, table, [0, 64, 128], 16, 128, status=False)
    out, _ = _run(np.zeros((0, 656), np.uint8), np.zeros((2, 0), np.int32), [0, 3, 5], 16, 5)
    assert (out == 0).all()


def test_rows_of_a_pool_past_4_gib():
    n_rows = 6_700_000   # 4.4 GB
    pool = torch.zeros((n_rows, 656), dtype=torch.uint8, device="cuda")
    tail = _pool(64, 3)
    pool[-64:] = torch.from_numpy(tail).cuda()
    table = torch.tensor([[n_rows // 64 - 1]], dtype=torch.int32, device="cuda")
    assert n_rows % 64 == 32   # the last whole page begins 96 rows before the end
    out = torch.empty((64, 576), dtype=torch.bfloat16, device="cuda")
    native.dsa_kv_gather(pool, table, torch.tensor([0, 64], dtype=torch.int32, device="cuda"), out, 64)
    want, _ = heads.kv_gather(tail, np.zeros((1, 1), np.int32), [0, 32], None, 64, 32)
    assert (out[:32] == 0).all()
    assert (np.abs(out[32:].double().cpu().numpy() - want) <= 1.01 * 2.0 ** -8 * np.abs(want)).all()


def test_what_the_insert_wrote_comes_back():
    """Within the insert's rounding (half an E4M3 step, 2^-4 of a value, or of 2^-6 of the block's largest / 448) and bf16's."""
    g = torch.Generator().manual_seed(4)
    n, page = 75, 16
    kv = torch.randn((n, 576), generator=g).to(torch.bfloat16)
    w = torch.ones(512).to(torch.bfloat16)
    table = torch.randperm(5, generator=g).to(torch.int32)[None]
    pos = torch.arange(n, dtype=torch.int32)
    slots = table[0, pos // page].long() * page + pos % page
    pool = torch.zeros((5 * page, 656), dtype=torch.uint8, device="cuda")
    native.dsa_kv_insert(kv.cuda(), pos.cuda(), slots.cuda(), w.cuda(), pool)
    out = torch.empty((n, 576), dtype=torch.bfloat16, device="cuda")
    native.dsa_kv_gather(pool, table.cuda(), torch.tensor([0, n], dtype=torch.int32, device="cuda"), out, page)
    x = kv.double()[:, :512]
    y = (x / (x.square().mean(dim=1, keepdim=True) + 1e-6).sqrt()).view(n, 4, 128)
    step = y.abs().amax(dim=2, keepdim=True) / 448 * 2.0 ** -6
    got = out.cpu().double()[:, :512].view(n, 4, 128)
    assert ((got - y).abs() <= 2.0 ** -4 * torch.maximum(y.abs(), step) + 1.1 * 2.0 ** -8 * y.abs() + 1e-6).all()
    ref = kv_insert(np.zeros((5 * page, 656), np.uint8), kv.view(torch.int16).numpy().view(np.uint16), pos.numpy(), slots.numpy(),
                    w.view(torch.int16).numpy().view(np.uint16))
    want, _ = heads.kv_gather(ref, table.numpy(), [0, n], None, page, n)
    assert (np.abs(out.double().cpu().numpy()[:, :512] - want[:, :512]) <= 1.01 * 2.0 ** -8 * np.abs(want[:, :512]) + 1e-6).all()


def test_graph_replayed_on_another_batch():
    pool, page = _pool(128, 5), 16
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    table = np.arange(8, dtype=np.int32).reshape(2, 4)
    pd, td, cu = t(pool), t(table), torch.tensor([0, 20, 60], dtype=torch.int32, device="cuda")
    out = torch.zeros((100, 576), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            native.dsa_kv_gather(pd, td, cu, out, page)
    cu.copy_(torch.tensor([3, 40, 100]))
    td.copy_(td.flip(0))
    g.replay()
    torch.cuda.synchronize()
    want, _ = heads.kv_gather(pool, table[::-1], [3, 40, 100], None, page, 100)
    got = out.double().cpu().numpy()
    assert (got[:3] == 0).all() and (np.abs(got[3:] - want[3:]) <= 1.01 * 2.0 ** -8 * np.abs(want[3:])).all()
