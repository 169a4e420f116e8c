"""The operators of a layer together, as a serving loop uses them.

Dense layers: the page map of a step gives positions, slots, tables and lengths; the heads of a packed qkv projection are normalised and
roped by them, the keys go into the paged 8-bit cache, and the queries of a group of requests behind one prompt attend.
Latent layers: a chunk's latent rows go into the cache, the whole context is read back, the up-projection expands it, and the chunk's
queries, roped by the same call, attend to it."""

import numpy as np
import pytest
import torch

from oracle import heads, paged
from test_kv8_attn_gpu import Case
from test_mla_prefill_gpu import Case as LatentCase
from top_sparse_mla_gb300 import native

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from top_sparse_mla_gb300.build import build
    build()
    native.library()


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_a_prompt_then_answers_that_share_it(dtype):
    page, h, g, d, n, cols, n_pages = 16, 2, 4, 128, 4, 16, 48
    t16 = torch.bfloat16 if dtype == "bf16" else torch.float16
    gen = torch.Generator(device="cuda").manual_seed(5)
    pools = [torch.full((n_pages, h, page, d), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.full((n_pages, h), float("nan"), device="cuda") for _ in range(2)]
    w = [(1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(t16) for _ in range(2)]
    free, table, ctx = _i32(np.random.default_rng(3).permutation(n_pages)), torch.full((n, cols), -1, dtype=torch.int32, device="cuda"), np.zeros(n, int)
    prompt = 75   # 4 whole pages are shared; every request has the rest of the prompt in a page of its own
    group, prefix = _i32([0, n]), _i32([prompt])
    # the prompt once, by request 0; then its pages in every table, and each request computes the prompt's rest and its own tokens
    for step, new in enumerate([[prompt // page * page, 0, 0, 0], [prompt % page + 2, prompt % page, prompt % page + 7, prompt % page + 1], [1] * n, [1, 3, 0, 1]]):
        if step == 1:
            table[1:] = table[0]
            ctx[:] = prompt // page * page
        total, n_tokens = sum(new), sum(new) + 2
        cu, kv = _i32(np.zeros(n + 1)), _i32(np.zeros(n))
        pos, slots, info = _i32(np.zeros(n_tokens)), torch.zeros(n_tokens, dtype=torch.int64, device="cuda"), _i32([0, 0])
        native.dsa_page_map(_i32(ctx), _i32(new), table, free, page, cu, kv, pos, slots, None, info)
        taken, status = info.tolist()
        assert status == 0
        free, ctx = free[taken:], ctx + np.array(new)
        qkv = torch.randn((n_tokens, h * g + 2 * h, d), generator=gen, device="cuda").to(t16)
        q, k, v = qkv[:, :h * g], qkv[:, h * g:h * g + h], qkv[:, h * g + h:]
        raw_q, raw_k = q.double().cpu().numpy(), k.double().cpu().numpy()
        native.dsa_qk_norm_rope(q, k, pos, w[0], w[1], q, k, native.dsa_qk_params_init(q, k))      # in place
        for got, raw, ww in ((q, raw_q, w[0]), (k, raw_k, w[1])):
            want, size = heads.norm_rope(raw, ww.double().cpu().numpy(), pos.tolist(), d)
            half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
            assert (np.abs(got.double().cpu().numpy() - want) <= half * np.abs(want) + 27 * 2.0 ** -24 * size + 2.0 ** -25).all()
        native.dsa_kv8_insert(k, v, slots, *pools, *scales)
        out, lse = torch.full((n_tokens, h * g, d), 7.0, dtype=t16, device="cuda"), torch.full((n_tokens, h * g), 7.0, device="cuda")
        p = native.dsa_kv8_params_init(q, pools[0], table, max_q_len=max(new))
        ws = torch.empty(native.dsa_kv8_prefix_workspace_size(p, 1), dtype=torch.uint8, device="cuda")
        native.dsa_kv8_prefix_attn_fwd(q, pools[0], pools[1], scales[0], scales[1], table, cu, kv, group, prefix, out, p, ws, lse=lse)
        assert native.dsa_sparse_attn_read_status(ws) == 0 and int(cu[-1]) == total
        c = Case.__new__(Case)
        c.h, c.g, c.d, c.dtype, c.kv = h, g, d, dtype, ctx + 16   # 16: the join of two parts
        c.check(out, lse, paged.kv8_attention(q.double().cpu().numpy(), pools[0].cpu().numpy(), pools[1].cpu().numpy(), scales[0].cpu().numpy(),
                                              scales[1].cpu().numpy(), table.cpu().numpy(), cu.cpu().numpy(), ctx, float(np.float32(d ** -0.5))))
        # and the plain call on the same tables: each is off by at most the bound, which c.check knows
        plain, plain_lse = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
        ws = torch.empty(native.dsa_kv8_attn_workspace_size(p), dtype=torch.uint8, device="cuda")
        native.dsa_kv8_attn_fwd(q, pools[0], pools[1], scales[0], scales[1], table, cu, kv, plain, p, ws, lse=plain_lse)
        assert torch.allclose(out[:total].float(), plain[:total].float(), rtol=2.0 ** -6, atol=2.0 ** -6)


def test_a_chunk_of_a_latent_layer_behind_its_context():
    page, h, n = 32, 4, 3
    gen = torch.Generator(device="cuda").manual_seed(6)
    lens = [(50, 130), (33, 33), (1, 200)]                       # chunk, and context with the chunk
    pages = [-(-kv // page) for _, kv in lens]
    order, table, at = np.random.default_rng(4).permutation(sum(pages) + 1), np.full((n, max(pages)), -1, np.int32), 0
    for r, used in enumerate(pages):
        table[r, :used] = order[at:at + used]
        at += used
    table = _i32(table)
    pool = torch.zeros(((sum(pages) + 1) * page, 656), dtype=torch.uint8, device="cuda")
    w = (1 + 0.1 * torch.randn(512, generator=gen, device="cuda")).to(torch.bfloat16)
    # the latent rows of contexts and chunks go in, at their positions
    cu, ck = np.concatenate([[0], np.cumsum([a for a, _ in lens])]), np.concatenate([[0], np.cumsum([b for _, b in lens])])
    pos = torch.cat([torch.arange(kv, dtype=torch.int32) for _, kv in lens]).cuda()
    req = torch.repeat_interleave(torch.arange(n), torch.tensor([kv for _, kv in lens])).cuda()
    slots = table[req, (pos // page).long()].long() * page + pos.long() % page
    rows = torch.randn((len(pos), 576), generator=gen, device="cuda").to(torch.bfloat16)
    native.dsa_kv_insert(rows, pos, slots, w, pool)
    # read back, and expanded for every head
    latent, status = torch.empty((len(pos), 576), dtype=torch.bfloat16, device="cuda"), _i32([0])
    native.dsa_kv_gather(pool, table, _i32(ck), latent, page, status=status)
    want, missing = heads.kv_gather(pool.cpu().numpy(), table.cpu().numpy(), ck, None, page, len(pos))
    assert status.item() == 0 and not missing
    assert (np.abs(latent.double().cpu().numpy() - want) <= 1.01 * 2.0 ** -8 * np.abs(want)).all()
    up = torch.randn((512, h * 256), generator=gen, device="cuda").div_(512 ** 0.5).to(torch.bfloat16)
    kv = (latent[:, :512] @ up).view(-1, h, 256)
    # the chunk's queries: the last 64 of their 192 dims turn
    q = torch.randn((cu[-1], h, 192), generator=gen, device="cuda").to(torch.bfloat16)
    q_pos = torch.cat([torch.arange(b - a, b, dtype=torch.int32) for a, b in lens]).cuda()
    native.dsa_qk_norm_rope(q, None, q_pos, None, None, q, None, native.dsa_qk_params_init(q, rotary_dim=64, rotary_start=128, interleaved=True))
    out, lse = torch.empty((cu[-1], h, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((cu[-1], h), device="cuda")
    p = native.dsa_mla_params_init(q, kv[:, :, :128], _i32(cu), max_q_len=50, max_kv_len=200)
    ws = torch.empty(native.dsa_mla_prefill_workspace_size(p), dtype=torch.uint8, device="cuda")
    native.dsa_mla_prefill_fwd(q, kv[:, :, :128], latent[:, 512:], kv[:, :, 128:], _i32(cu), _i32(ck), out, p, ws, lse=lse)
    assert native.dsa_sparse_attn_read_status(ws) == 0
    c = LatentCase.__new__(LatentCase)
    c.lens, c.h, c.dtype, c.scale, c.cu, c.ck = lens, h, "bf16", 192 ** -0.5, cu, ck
    c.q, c.up, c.latent = q.cpu(), kv.cpu(), latent.cpu()
    c.check(out, lse)
