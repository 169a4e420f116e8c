"""The page map's CUDA path (include/dsa_page_map.h) against the oracle (oracle/paged.py):
every integer equal, and every byte that the call does not own left as it was."""

import numpy as np
import pytest
import torch

from oracle import paged
from top_sparse_mla_gb300 import native

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from top_sparse_mla_gb300.build import build
    build()
    native.library()


def _dev(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def _run(ctx, new, table, free, page, n_tokens, pitch=0, req=True, stream=None):
    n, cols = table.shape
    buf = torch.full((max(n, 1), cols + pitch), -77, dtype=torch.int32, device="cuda")
    buf[:n, :cols] = _dev(table)
    t = buf[:n, :cols]
    guard = 3   # entries behind each output that must stay
    out = {"cu": torch.full((n + 1 + guard,), -5, dtype=torch.int32, device="cuda"),
           "kv": torch.full((n + guard,), -5, dtype=torch.int32, device="cuda"),
           "pos": torch.full((n_tokens + guard,), -5, dtype=torch.int32, device="cuda"),
           "slots": torch.full((n_tokens + guard,), -5, dtype=torch.int64, device="cuda"),
           "req": torch.full((n_tokens + guard,), -5, dtype=torch.int32, device="cuda"),
           "info": torch.full((2 + guard,), -5, dtype=torch.int32, device="cuda")}
    o = {k: v[:v.numel() - guard] for k, v in out.items()}
    native.dsa_page_map(_dev(ctx), _dev(new), t, _dev(free), page, o["cu"], o["kv"], o["pos"], o["slots"],
                        o["req"] if req else None, o["info"], stream=stream)
    torch.cuda.synchronize()
    for v in out.values():
        assert (v[-guard:] == -5).all()
    assert (buf[:n, cols:] == -77).all() and (buf[n:] == -77).all()
    return [t.cpu().numpy()] + [o[k].cpu().numpy() for k in ("cu", "kv", "pos", "slots", "req", "info")]


def _check(ctx, new, table, free, page, n_tokens, **kw):
    want = paged.page_map(ctx, new, table, free, page, n_tokens)
    got = _run(ctx, new, table, free, page, n_tokens, **kw)
    for name, a, b in zip(("table", "cu", "kv_lens", "positions", "slots", "token_req", "info"), got, want):
        if name == "token_req" and not kw.get("req", True):
            continue
        assert np.array_equal(a, b), name
    return want


def _case(seed, n, ctx_max, new_max, page, spare=4, cols_more=0):
    rng = np.random.default_rng(seed)
    ctx, new = rng.integers(0, ctx_max + 1, n), rng.integers(0, new_max + 1, n)
    old, need = -(-ctx // page), -(-(ctx + new) // page)
    cols = int(max(need.max() if n else 1, 1)) + cols_more
    ids = rng.permutation(int(old.sum() + (need - old).sum()) + spare).astype(np.int32)
    table = np.full((n, cols), -9, np.int32)
    at = 0
    for r in range(n):
        table[r, :old[r]] = ids[at:at + old[r]]
        at += old[r]
    return ctx, new, table, ids[at:], page, int(new.sum())


@pytest.mark.parametrize("n,ctx_max,new_max,page,pad", [
    (1, 0, 1, 16, 0), (1, 5, 0, 16, 0), (3, 40, 1, 16, 2), (17, 1000, 1, 64, 0), (33, 300, 500, 32, 7), (2, 10, 3000, 1, 0),
    (513, 100, 3, 48, 1), (2000, 3000, 1, 16, 96), (8192, 20, 2, 8, 0), (6144, 50, 1, 128, 5)])
def test_random_batches(n, ctx_max, new_max, page, pad):
    ctx, new, table, free, page, t = _case(n + new_max, n, ctx_max, new_max, page)
    want = _check(ctx, new, table, free, page, t + pad)
    assert want[-1][1] == 0


def test_a_table_with_a_row_pitch_and_no_token_requests():
    ctx, new, table, free, page, t = _case(5, 40, 200, 30, 16, cols_more=3)
    _check(ctx, new, table, free, page, t + 4, pitch=5, req=False)


def test_no_requests_and_no_tokens():
    empty = np.zeros((0, 4), np.int32)
    _check([], [], empty, [], 16, 9)
    _check([], [], empty, [], 16, 0)
    _check([3, 0], [0, 0], np.array([[1], [2]], np.int32), [], 16, 0)


def test_negative_lengths_count_as_zero():
    _check([-4, 7, -1], [3, -2, -2 ** 31], np.array([[-1, -1], [5, -1], [-1, -1]], np.int32), [8, 9], 8, 5)


def test_out_of_pages_full_tables_and_full_batches_are_reported():
    ctx, new, table, free, page, t = _case(8, 50, 60, 40, 16, spare=0)
    want = _check(ctx, new, table, free[:len(free) // 2], page, t)
    assert want[-1][1] == native.DSA_STATUS_OUT_OF_PAGES
    holes = free.copy()
    holes[::3] = -1
    assert _check(ctx, new, table, holes, page, t)[-1][1] == native.DSA_STATUS_OUT_OF_PAGES
    assert _check(ctx, new, table, free, page, t // 2)[-1][1] == native.DSA_STATUS_TOKENS_FULL
    assert _check(ctx, new, np.ascontiguousarray(table[:, :3]), free, page, t)[-1][1] & native.DSA_STATUS_TABLE_FULL
    # a request whose half-filled page is missing from the table
    assert _check([3], [2], np.array([[-1]], np.int32), [], 8, 2)[-1][1] == native.DSA_STATUS_OUT_OF_PAGES


def test_lengths_near_the_type_s_end():
    big = 2 ** 31 - 1
    got = _run([big - 2, big], [1, big], np.array([[4, 5], [6, 7]], np.int32), [], 1 << 20, 6)
    # far past the table's two columns: no slots, and the lengths stop at 2^31 - 1
    assert got[1].tolist() == [0, 1, 6] and got[2].tolist() == [big - 1, big]
    assert got[3].tolist() == [big - 2, big, big, big, big, big] and (got[4] == -1).all()
    assert got[6][1] == native.DSA_STATUS_TABLE_FULL | native.DSA_STATUS_TOKENS_FULL


def test_slots_past_32_bits():
    got = _run([0], [3], np.array([[-1]], np.int32), [2 ** 31 - 1], 64, 3)
    assert got[4].tolist() == [(2 ** 31 - 1) * 64 + i for i in range(3)]


def test_replayed_from_a_graph_on_another_stream():
    ctx, new, table, free, page, t = _case(21, 64, 500, 1, 16)
    want = paged.page_map(ctx, new, table, free, page, t)
    args = dict(ctx=_dev(ctx), new=_dev(new), table=_dev(table), free=_dev(free), cu=_dev(np.zeros(65)), kv=_dev(np.zeros(64)),
                pos=_dev(np.zeros(t)), slots=_dev(np.zeros(t), torch.int64), req=_dev(np.zeros(t)), info=_dev([0, 0]))

    def call():
        a = args
        native.dsa_page_map(a["ctx"], a["new"], a["table"], a["free"], page, a["cu"], a["kv"], a["pos"], a["slots"],
                            a["req"], a["info"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in ("cu", "kv", "pos", "slots", "req", "info"):
        args[k].fill_(-3)
    args["table"].copy_(_dev(table))
    graph.replay()
    torch.cuda.synchronize()
    for name, w in zip(("table", "cu", "kv", "pos", "slots", "req", "info"), want):
        assert np.array_equal(args[name].cpu().numpy(), w), name
