"""The paged-cache operators together, as a serving loop uses them: the page map of a step
gives positions, slots, tables and lengths; the insert and the attention take them.  Also
the page map in front of the latent path: its positions and slots drive dsa_kv_insert and
the rows that dsa_sparse_attn_fwd gathers."""

import numpy as np
import pytest
import torch

import oracle
from oracle import paged
from oracle.kv_insert import kv_insert
from top_sparse_mla_gb300 import native
from top_sparse_mla_gb300 import workloads as W
from test_kv8_attn_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from top_sparse_mla_gb300.build import build
    build()
    native.library()


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_prefill_then_decode_steps(dtype):
    page, h, g, d, n, cols = 16, 2, 4, 64, 5, 12
    n_pages = 60
    rng = np.random.default_rng(1)
    pools = [torch.full((n_pages, h, page, d), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.full((n_pages, h), float("nan"), device="cuda") for _ in range(2)]
    ref = [np.full((n_pages, h, page, d), 0x7F, np.uint8), np.full((n_pages, h), np.nan, np.float32)]
    ref += [ref[0].copy(), ref[1].copy()]
    table = torch.full((n, cols), -1, dtype=torch.int32, device="cuda")
    free = rng.permutation(n_pages).astype(np.int32)
    ctx = np.zeros(n, int)
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float16
    for step, new in enumerate([[40, 1, 0, 100, 17], [1, 1, 33, 1, 1], [1, 2, 1, 0, 4], [1, 1, 1, 1, 1]]):
        total, n_tokens = sum(new), sum(new) + 3          # a padded batch
        cu, kv, req = _i32(np.zeros(n + 1)), _i32(np.zeros(n)), _i32(np.zeros(n_tokens))
        pos, slots, info = _i32(np.zeros(n_tokens)), torch.zeros(n_tokens, dtype=torch.int64, device="cuda"), _i32([0, 0])
        native.dsa_page_map(_i32(ctx), _i32(new), table, _i32(free), page, cu, kv, pos, slots, req, info)
        k, v, q = (torch.from_numpy(rng.standard_normal((n_tokens, hh, d)) * m).to(tdt).cuda()
                   for hh, m in ((h, 1.0), (h, 3.0), (h * g, 2.0)))
        native.dsa_kv8_insert(k, v, slots, pools[0], pools[1], scales[0], scales[1])
        out = torch.full((n_tokens, h * g, d), 7.0, dtype=tdt, device="cuda")
        lse = torch.full((n_tokens, h * g), 7.0, device="cuda")
        p = native.dsa_kv8_params_init(q, pools[0], table, max_q_len=max(new))
        ws = torch.empty(native.dsa_kv8_attn_workspace_size(p), dtype=torch.uint8, device="cuda")
        native.dsa_kv8_attn_fwd(q, pools[0], pools[1], scales[0], scales[1], table, cu, kv, out, p, ws, lse=lse)
        taken, status = info.tolist()
        assert status == 0 and native.dsa_sparse_attn_read_status(ws) == 0
        free = free[taken:]
        ctx = ctx + np.array(new)
        assert kv.tolist() == ctx.tolist() and int(cu[-1]) == total
        sl = slots.cpu().numpy()
        for i, x in ((0, k), (2, v)):
            ref[i], ref[i + 1] = paged.kv8_insert(ref[i], ref[i + 1], x.double().cpu().numpy(), sl)
        assert np.array_equal(pools[0].cpu().numpy(), ref[0]) and np.array_equal(pools[1].cpu().numpy(), ref[2])
        live = ~np.isnan(ref[1])
        assert np.array_equal(scales[0].cpu().numpy()[live], ref[1][live])
        c = Case.__new__(Case)
        c.h, c.g, c.d, c.dtype, c.kv = h, g, d, dtype, ctx
        c.check(out, lse, paged.kv8_attention(q.double().cpu().numpy(), ref[0], ref[2], ref[1], ref[3], table.cpu().numpy(),
                                              cu.cpu().numpy(), ctx, float(np.float32(d ** -0.5))))


def test_the_map_drives_the_latent_insert_and_its_attention():
    import parity
    w0 = W.make("tiny")
    n_rows, page = w0.kv_cmp.shape[0], 16
    rng = np.random.default_rng(2)
    n = 3
    new = np.array([n_rows // page * page - 200, 150, 50])
    cols = 40
    table = torch.full((n, cols), -1, dtype=torch.int32, device="cuda")
    free = _i32(rng.permutation(n_rows // page))
    t = int(new.sum())
    cu, kv, info = _i32(np.zeros(n + 1)), _i32(np.zeros(n)), _i32([0, 0])
    pos, slots = _i32(np.zeros(t)), torch.zeros(t, dtype=torch.int64, device="cuda")
    native.dsa_page_map(_i32([0] * n), _i32(new), table, free, page, cu, kv, pos, slots, None, info)
    # 312, 150 and 50 tokens need 34 pages and the pool has 32: the last tokens have slot -1
    assert n_rows == 512 and info.tolist() == [32, native.DSA_STATUS_OUT_OF_PAGES]
    bits = oracle.codecs.bf16_encode(rng.standard_normal((t, 576)))
    wn = oracle.codecs.bf16_encode(1.0 + 0.1 * rng.standard_normal(512))
    pool = torch.from_numpy(w0.kv_cmp.copy()).cuda()
    sl, ps = slots.cpu().numpy(), pos.cpu().numpy()
    native.dsa_kv_insert(torch.from_numpy(bits.view(np.int16)).cuda(), pos, slots,
                         torch.from_numpy(wn.view(np.int16)).cuda(), pool)
    got = pool.cpu().numpy()
    want = kv_insert(w0.kv_cmp, bits, ps, sl, wn)
    written = sl[sl >= 0]
    others = np.setdiff1d(np.arange(n_rows), written)
    assert np.array_equal(got[others], w0.kv_cmp[others]) and np.array_equal(got[written, :512], want[written, :512])
    idx = w0.indices.copy()
    idx[:, w0.n_swa_cols:] = rng.choice(written, idx[:, w0.n_swa_cols:].shape)
    w1 = W.Workload(name="tiny_mapped", q=w0.q, norm_w=w0.norm_w, kv_swa=w0.kv_swa, kv_cmp=got, indices=idx,
                    topk_length=w0.topk_length, positions=w0.positions, n_swa_cols=w0.n_swa_cols, seed=w0.seed)
    parity.compare(parity.run_gpu(w1), parity.run_oracle(w1), label="attention on rows of a page map")
