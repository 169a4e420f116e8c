"""The binding's checks of the tensors that the head norm, the cache read-back and the two attentions beside the caches take: one wrong
property at a time, the argument named in the error, and nothing written.  On the CPU the check of the device is replaced, so that the
others are reached, and the launching entry points by ones that must not be called; on a GPU everything is as a caller has it."""

import pytest
import torch

from test_paged_binding import COLS, D, HQ, N, PAGE, PAGES, Reached, T, _bad_cache, _cache, _check, _wide
from top_sparse_mla_gb300 import native

LAUNCH = ("dsa_qk_norm_rope", "dsa_kv_gather", "dsa_mla_prefill_fwd", "dsa_kv8_prefix_attn_fwd")


@pytest.fixture(params=["cpu", pytest.param("cuda", marks=pytest.mark.gpu)])
def device(request, monkeypatch):
    from top_sparse_mla_gb300.build import build
    build()
    if request.param == "cpu":
        native._bind_torch()
        monkeypatch.setattr(native, "_device", lambda where, x: -1)
        monkeypatch.setattr(native, "_stream", lambda stream, dev: 0)
        real = native.library()

        class Library:
            def __getattr__(self, name):
                if name not in LAUNCH:
                    return getattr(real, name)

                def call(*args):
                    raise Reached(name)
                return call

        monkeypatch.setattr(native, "library", lambda *a: Library())
    return request.param


def _other(dtype):
    return torch.float16 if dtype == torch.bfloat16 else torch.bfloat16


def _bad_heads(name, other):
    return [(name, lambda x: x[:-1]), (name, lambda x: x[:, :-1]), (name, lambda x: x[:, :, :32]), (name, lambda x: x[0]), (name, _wide),
            (name, lambda x: x.to(other)), (name, torch.Tensor.float)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_norm_rope(device, dtype):
    q, k = torch.ones((T, 4, 64), dtype=dtype, device=device), torch.ones((T, 2, 64), dtype=dtype, device=device)
    p = native.dsa_qk_params_init(q, k, rotary_dim=32)
    w = torch.ones(64, dtype=dtype, device=device)
    good = dict(q=q, k=k, positions=torch.arange(T, dtype=torch.int32, device=device), q_weight=w, k_weight=w.clone(), q_out=q * 7, k_out=k * 7, p=p)
    bad = [b for name in ("q", "k", "q_out", "k_out") for b in _bad_heads(name, _other(dtype))]
    for name in ("q_weight", "k_weight"):
        bad += [(name, torch.Tensor.float), (name, lambda x: x[:-1]), (name, _wide), (name, lambda x: x[None])]
    bad += [("positions", torch.Tensor.long), ("positions", lambda x: x[:-1]), ("positions", _wide), ("k", lambda x: None), ("k_out", lambda x: None)]
    if device == "cuda":
        bad += [(name, torch.Tensor.cpu) for name in good if name not in ("p", "q")]
    _check(native.dsa_qk_norm_rope, good, bad, ("q_out", "k_out"), device)
    for wrong in ((q.float(), k), (q[0], k), (q, k.float()), (q, k[:-1]), (q, k[:, :, :32])):
        with pytest.raises(native.DsaError):
            native.dsa_qk_params_init(*wrong)
    assert native.dsa_qk_params_init(q).h_k == 0


def test_gather(device):
    i32 = dict(dtype=torch.int32, device=device)
    good = dict(pool=torch.zeros((PAGES * PAGE, 656), dtype=torch.uint8, device=device), block_table=torch.zeros((N, COLS), **i32),
                cu_rows=torch.tensor([0, 2, 3, 5], **i32), out=torch.full((T, 576), 7.0, dtype=torch.bfloat16, device=device), page_size=PAGE,
                lens=torch.ones(N, **i32), status=torch.zeros(1, **i32))
    bad = [("pool", lambda x: x[:, :640]), ("pool", _wide), ("pool", lambda x: x.view(torch.int8)), ("pool", lambda x: x[0]),
           ("cu_rows", torch.Tensor.long), ("cu_rows", lambda x: x[:-1]), ("cu_rows", _wide), ("lens", torch.Tensor.long), ("lens", lambda x: x[:-1]),
           ("lens", _wide), ("out", torch.Tensor.half), ("out", lambda x: x[:, :512]), ("out", _wide), ("out", lambda x: x[0]),
           ("out", lambda x: x[:1].expand(T, -1)), ("status", torch.Tensor.long), ("block_table", torch.Tensor.long), ("block_table", lambda x: x[0]),
           ("block_table", lambda x: x.t().contiguous().t())]
    if device == "cuda":
        bad += [(name, torch.Tensor.cpu) for name in good if name not in ("page_size", "pool")]
    _check(native.dsa_kv_gather, good, bad, ("out", "status"), device)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_latent_attention(device, dtype):
    def ones(*shape):
        return torch.ones(shape, dtype=dtype, device=device)

    q, k, cu = ones(T, HQ, 192), ones(7, HQ, 128), torch.tensor([0, 1, 3, 5], dtype=torch.int32, device=device)
    p = native.dsa_mla_params_init(q, k, cu)
    good = dict(q=q, k_nope=k, k_rope=ones(7, 64), v=ones(7, HQ, 128), cu_q=cu, cu_kv=cu + torch.arange(4, dtype=torch.int32, device=device) // 2,
                out=ones(T, HQ, 128) * 7, p=p, workspace=torch.zeros(native.dsa_mla_prefill_workspace_size(p, 152), dtype=torch.uint8, device=device),
                lse=torch.full((T, HQ), 7.0, device=device))
    other = _other(dtype)
    bad = [b for name in ("q", "k_nope", "v", "out") for b in _bad_heads(name, other)]
    bad += [("k_rope", lambda x: x[:-1]), ("k_rope", lambda x: x[:, :32]), ("k_rope", _wide), ("k_rope", lambda x: x.to(other)), ("k_rope", lambda x: x[0])]
    for name in ("cu_q", "cu_kv"):
        bad += [(name, torch.Tensor.long), (name, lambda x: x[:-1]), (name, _wide)]
    bad += [("lse", torch.Tensor.half), ("lse", lambda x: x[:-1]), ("lse", _wide), ("workspace", _wide)]
    if device == "cuda":
        bad += [(name, torch.Tensor.cpu) for name in good if name not in ("p", "q")]
    _check(native.dsa_mla_prefill_fwd, good, bad, ("out", "lse", "workspace"), device)
    if device == "cuda":
        with pytest.raises(native.DsaError) as e:
            native.dsa_mla_prefill_fwd(**dict(good, workspace=good["workspace"][:256]))
        assert e.value.code == native.DSA_ERR_WORKSPACE_TOO_SMALL
    for wrong in ((q.float(), k, cu), (q[:, :, :128], k, cu), (q, k[:, :2], cu), (q, k.to(other), cu), (q, k, cu[:0])):
        with pytest.raises(native.DsaError):
            native.dsa_mla_params_init(*wrong)
    with pytest.raises(native.DsaError):
        native.dsa_mla_params_init(q, k, cu, window=3)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_prefix_attention(device, dtype):
    cache = _cache(device)
    i32 = dict(dtype=torch.int32, device=device)
    q, table = torch.ones((T, HQ, D), dtype=dtype, device=device), torch.zeros((N, COLS), **i32)
    p = native.dsa_kv8_params_init(q, cache["k_pool"], table, max_q_len=2)
    good = dict(q=q, block_table=table, cu_q=torch.tensor([0, 1, 3, 5], **i32), kv_lens=torch.full((N,), 20, **i32),
                cu_groups=torch.tensor([0, 2, 3], **i32), prefix_lens=torch.full((2,), 16, **i32), out=torch.full_like(q, 7.0), p=p,
                workspace=torch.zeros(native.dsa_kv8_prefix_workspace_size(p, 2, 152), dtype=torch.uint8, device=device),
                lse=torch.full((T, HQ), 7.0, device=device), **cache)
    bad = _bad_cache(device) + [b for name in ("q", "out") for b in _bad_heads(name, _other(dtype))]
    for name in ("cu_q", "kv_lens", "cu_groups", "prefix_lens"):
        bad += [(name, torch.Tensor.long), (name, _wide)]
    bad += [("cu_q", lambda x: x[:-1]), ("kv_lens", lambda x: x[:-1]), ("cu_groups", lambda x: x[:-1]), ("cu_groups", lambda x: x[None]),
            ("prefix_lens", lambda x: x[None]), ("lse", torch.Tensor.half), ("lse", lambda x: x[:-1]), ("block_table", torch.Tensor.long),
            ("block_table", lambda x: x[:-1]), ("workspace", _wide)]
    if device == "cuda":
        bad += [(name, torch.Tensor.cpu) for name in good if name not in ("p", "q")]
    _check(native.dsa_kv8_prefix_attn_fwd, good, bad, ("out", "lse", "workspace"), device)
    if device == "cuda":
        with pytest.raises(native.DsaError) as e:
            native.dsa_kv8_prefix_attn_fwd(**dict(good, workspace=good["workspace"][:256]))
        assert e.value.code == native.DSA_ERR_WORKSPACE_TOO_SMALL
