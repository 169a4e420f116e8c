"""The binding's checks of the paged-cache operators' tensors: one wrong property at a time, the argument named in the error, and
nothing written.  On the CPU the check of the device is replaced, so that the others are reached, and the library by one that
must not be called; on a GPU everything is as a caller has it."""

import pytest
import torch

from top_sparse_mla_gb300 import native

N, T, COLS, PAGES, H, HQ, PAGE, D = 3, 5, 4, 6, 2, 4, 16, 64


class Reached(Exception):
    """The arguments passed the binding's checks."""


class NoLibrary:
    def __getattr__(self, name):
        def call(*args):
            raise Reached(name)
        return call


@pytest.fixture(params=["cpu", pytest.param("cuda", marks=pytest.mark.gpu)])
def device(request, monkeypatch):
    if request.param == "cpu":
        native._bind_torch()
        monkeypatch.setattr(native, "_device", lambda where, x: -1)
        monkeypatch.setattr(native, "_stream", lambda stream: 0)
        real = native.library

        class Params(NoLibrary):
            dsa_kv8_params_init = property(lambda self: real().dsa_kv8_params_init)
            dsa_kv8_attn_workspace_size = property(lambda self: real().dsa_kv8_attn_workspace_size)
            dsa_error_string = property(lambda self: real().dsa_error_string)

        from top_sparse_mla_gb300.build import build
        build()
        monkeypatch.setattr(native, "library", lambda *a: Params())
    else:
        from top_sparse_mla_gb300.build import build
        build()
    return request.param


def _wide(x):
    """x as every second element of a tensor's last dimension."""
    return torch.stack([x, x], dim=-1).flatten(-2)[..., ::2]


def _check(call, good, bad, outputs, device):
    """call(**good) is accepted; with any of `bad`'s changes it is refused with the argument's name in the error."""
    if device == "cpu":
        with pytest.raises(Reached):
            call(**good)
    else:
        call(**good)
        torch.cuda.synchronize()
    for name, change in bad:
        args = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in good.items()}
        args[name] = change(args[name])
        before = {k: args[k].clone() for k in outputs if args[k] is not None}
        with pytest.raises(native.DsaError) as e:
            call(**args)
        assert e.value.code == native.DSA_ERR_INVALID_ARG and name in str(e.value), (name, str(e.value))
        if device == "cuda":
            torch.cuda.synchronize()
        for k, v in before.items():
            assert torch.equal(args[k], v), f"{k} was written with a bad {name}"


def test_page_map(device):
    def i32(*shape):
        return torch.zeros(shape, dtype=torch.int32, device=device)

    good = dict(ctx_lens=i32(N), new_lens=i32(N) + 1, block_table=i32(N, COLS), free_pages=i32(9), page_size=PAGE, cu_new=i32(N + 1),
                kv_lens=i32(N), positions=i32(T), slots=torch.zeros(T, dtype=torch.int64, device=device), token_req=i32(T), info=i32(2))
    bad = [(name, change) for name in ("ctx_lens", "new_lens", "free_pages", "cu_new", "kv_lens", "positions", "token_req", "info")
           for change in (torch.Tensor.long, _wide)]
    bad += [(name, lambda x: x[:-1]) for name in ("new_lens", "cu_new", "kv_lens", "positions", "token_req", "info")]
    bad += [(name, lambda x: torch.cat([x, x])) for name in ("new_lens", "cu_new", "kv_lens", "positions", "token_req", "info")]
    bad += [("slots", torch.Tensor.int), ("slots", _wide), ("block_table", torch.Tensor.long), ("block_table", lambda x: x[:-1]),
            ("block_table", lambda x: x.t().contiguous().t()), ("block_table", lambda x: x[:1].expand(N, -1)),
            ("block_table", lambda x: x[0])]
    if device == "cuda":
        bad += [(name, torch.Tensor.cpu) for name in good if name not in ("page_size", "ctx_lens")]
    _check(native.dsa_page_map, good, bad, ("block_table", "cu_new", "kv_lens", "positions", "slots", "token_req", "info"), device)


def _cache(device):
    return dict(k_pool=torch.zeros((PAGES, H, PAGE, D), dtype=torch.uint8, device=device),
                v_pool=torch.zeros((PAGES, H, PAGE, D), dtype=torch.uint8, device=device),
                k_scale=torch.ones((PAGES, H), device=device), v_scale=torch.ones((PAGES, H), device=device))


def _bad_cache(device):
    bad = [("v_pool", lambda x: x[:-1]), ("v_pool", lambda x: x.view(torch.int8)), ("k_pool", lambda x: x.view(torch.int8)),
           ("v_pool", lambda x: x.transpose(1, 2).contiguous().transpose(1, 2)), ("k_pool", _wide), ("v_pool", _wide),
           ("k_pool", lambda x: x[0])]
    for name in ("k_scale", "v_scale"):
        bad += [(name, torch.Tensor.double), (name, torch.Tensor.half), (name, lambda x: x[:-1]), (name, lambda x: x[:, :1]),
                (name, _wide), (name, lambda x: x.t().contiguous().t())]
    if device == "cuda":
        bad += [(name, torch.Tensor.cpu) for name in ("k_pool", "v_pool", "k_scale", "v_scale")]
    return bad


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_insert(device, dtype):
    good = dict(k=torch.ones((T, H, D), dtype=dtype, device=device), v=torch.ones((T, H, D), dtype=dtype, device=device),
                slots=torch.arange(T, device=device), status=torch.zeros(1, dtype=torch.int32, device=device), **_cache(device))
    other = torch.float16 if dtype == torch.bfloat16 else torch.bfloat16
    bad = _bad_cache(device) + [("slots", torch.Tensor.int), ("slots", _wide), ("status", torch.Tensor.long), ("k", torch.Tensor.float),
                                ("v", lambda x: x.to(other))]
    for name in ("k", "v"):
        bad += [(name, lambda x: x[:-1]), (name, lambda x: x[:, :1]), (name, lambda x: x[:, :, :32]), (name, lambda x: x[0]),
                (name, lambda x: torch.cat([x, x])), (name, _wide), (name, lambda x: x.transpose(1, 2).contiguous().transpose(1, 2))]
    if device == "cuda":
        bad += [(name, torch.Tensor.cpu) for name in ("v", "slots", "status")]
    _check(native.dsa_kv8_insert, good, bad, ("k_pool", "v_pool", "k_scale", "v_scale", "status"), device)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_attention(device, dtype):
    cache = _cache(device)
    q = torch.ones((T, HQ, D), dtype=dtype, device=device)
    table = torch.zeros((N, COLS), dtype=torch.int32, device=device)
    p = native.dsa_kv8_params_init(q, cache["k_pool"], table, max_q_len=2)
    good = dict(q=q, block_table=table, cu_q=torch.tensor([0, 1, 3, 5], dtype=torch.int32, device=device),
                kv_lens=torch.full((N,), 7, dtype=torch.int32, device=device), out=torch.full_like(q, 7.0), p=p,
                workspace=torch.zeros(native.dsa_kv8_attn_workspace_size(p, 152), dtype=torch.uint8, device=device),
                lse=torch.full((T, HQ), 7.0, device=device), **cache)
    other = torch.float16 if dtype == torch.bfloat16 else torch.bfloat16
    bad = [b for b in _bad_cache(device)]
    for name in ("q", "out"):
        bad += [(name, lambda x: x[:-1]), (name, lambda x: x[:, :-1]), (name, lambda x: x[:, :, :32]), (name, lambda x: x[0]), (name, _wide)]
    bad += [("q", lambda x: x.to(other)), ("q", torch.Tensor.float), ("out", lambda x: x.to(other)), ("out", torch.Tensor.float)]
    for name in ("cu_q", "kv_lens"):
        bad += [(name, torch.Tensor.long), (name, lambda x: x[:-1]), (name, _wide), (name, lambda x: torch.cat([x, x]))]
    bad += [("lse", torch.Tensor.half), ("lse", lambda x: x[:-1]), ("lse", lambda x: x[:, :1]), ("lse", _wide),
            ("block_table", torch.Tensor.long), ("block_table", lambda x: x[:-1]), ("block_table", lambda x: x[:, :-1]),
            ("block_table", lambda x: x.t().contiguous().t()), ("block_table", lambda x: x[:1].expand(N, -1)), ("workspace", _wide)]
    if device == "cuda":
        bad += [(name, torch.Tensor.cpu) for name in ("block_table", "cu_q", "kv_lens", "out", "workspace", "lse")]
    _check(native.dsa_kv8_attn_fwd, good, bad, ("out", "lse", "workspace"), device)


def test_tensors_of_the_host_are_refused_as_such():
    """Without a replaced check: the first tensor is not on the current CUDA device."""
    if not torch.cuda.is_available():
        k = torch.ones((T, H, D), dtype=torch.bfloat16)
        with pytest.raises(native.DsaError, match="current CUDA device"):
            native.dsa_kv8_insert(k, k, torch.arange(T), **_cache("cpu"))
