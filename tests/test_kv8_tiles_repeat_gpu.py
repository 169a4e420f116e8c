"""The attention over the paged 8-bit cache on many tiles, over and over: the same inputs give the same bits.  (A block's codes have one
buffer; where it is filled again before all of them were read, some rows of a tile's values are the next block's, once in some ten
thousand tiles.)"""

import pytest
import torch

from top_sparse_mla_gb300 import native

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from top_sparse_mla_gb300.build import build
    build()
    native.library()


# (requests, shared tokens or None, queries, own tokens behind the shared ones)
MIXED = [(18, None, 2, 270), (2, 221, 30, 120), (13, 693, 5, 150), (10, 80, 30, 160), (3, 642, 200, 330), (3, 73, 200, 300), (23, 391, 1, 90)]
CHUNKS = [(6, None, 300, 900), (4, 512, 200, 260)]


@pytest.mark.parametrize("d,h,g,page,dtype,batch", [(128, 8, 16, 128, torch.bfloat16, MIXED), (64, 4, 16, 16, torch.float16, MIXED),
                                                    (128, 8, 8, 64, torch.float16, CHUNKS)], ids=["mixed", "mixed, 64", "chunks"])
def test_the_same_bits_every_time(d, h, g, page, dtype, batch):
    gen = torch.Generator().manual_seed(7)
    lens, rows, cu_groups, prefix, pages = [], [], [], [], 0
    for n, shared, q, own in batch:
        common = list(range(pages, pages + (shared or 0) // page))
        pages += len(common)
        if shared is not None:
            cu_groups = cu_groups or [len(lens)]
            prefix.append(shared)
        for i in range(n):
            kv = (shared or 0) + own + 7 * i
            mine = -(-kv // page) - len(common)
            rows.append(common + list(range(pages, pages + mine)))
            pages += mine
            lens.append((q, kv))
        if shared is not None:
            cu_groups.append(len(lens))
    order = torch.randperm(pages, generator=gen).to(torch.int32)
    table = torch.full((len(lens), max(map(len, rows))), -1, dtype=torch.int32)
    for r, row in enumerate(rows):
        table[r, :len(row)] = order[row]

    def pool():
        sign = torch.randint(0, 2, (pages, h, page, d), generator=gen) * 128
        return (torch.randint(0, 0x78, (pages, h, page, d), generator=gen) + sign).to(torch.uint8).cuda()

    k_pool, v_pool = pool(), pool()
    k_scale = torch.full((pages, h), 2.0 ** -7, device="cuda")
    v_scale = torch.exp2(torch.randint(-8, -4, (pages, h), generator=gen).float()).cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table, kv, cu = table.cuda(), i32([b for _, b in lens]), i32([0] + torch.tensor([a for a, _ in lens]).cumsum(0).tolist())
    q = torch.randn((int(cu[-1]), h * g, d), generator=gen).to(dtype).cuda()
    p = native.dsa_kv8_params_init(q, k_pool, table, max_q_len=max(a for a, _ in lens))
    args = (q, k_pool, v_pool, k_scale, v_scale, table, cu, kv)
    plain_ws = torch.empty(native.dsa_kv8_attn_workspace_size(p), dtype=torch.uint8, device="cuda")
    ws = torch.empty(native.dsa_kv8_prefix_workspace_size(p, len(prefix)), dtype=torch.uint8, device="cuda")
    cu_groups, prefix = i32(cu_groups), i32(prefix)

    def plain(out, lse):
        native.dsa_kv8_attn_fwd(*args, out, p, plain_ws, lse=lse)
        return plain_ws

    def shared(out, lse):
        native.dsa_kv8_prefix_attn_fwd(*args, cu_groups, prefix, out, p, ws, lse=lse)
        return ws

    results = []
    for call in (plain, shared):
        want, want_l = torch.empty_like(q), torch.empty((len(q), h * g), device="cuda")
        out, lse = torch.empty_like(q), torch.empty_like(want_l)
        call(want, want_l)
        other = torch.zeros((), dtype=torch.int64, device="cuda")
        for _ in range(400):
            status = call(out, lse)
            other += (out != want).any() | (lse != want_l).any()
        assert native.dsa_sparse_attn_read_status(status) == 0
        assert int(other) == 0, f"{call.__name__}: {int(other)} of 400 runs differ"
        results.append((want.double(), want_l.double()))
    # Both calls are within their bounds of the same numbers: half a step of the result, 2^-11 of mass for the weights, and here at most
    # a quarter of that for the rest; mass is at most the largest value, 448 * 2^-5.
    half = 2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -11
    (a, al), (b, bl) = results
    assert bool(((a - b).abs() <= 2 * half * b.abs() + 2 * 1.25 * 2.0 ** -11 * 14).all())
    assert bool(((al - bl).abs() <= 1e-4).all())
