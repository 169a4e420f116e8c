"""Host-side checks of the paged-cache entry points (no GPU): arguments are refused before
anything touches a GPU, by the C ABI and by the binding."""

import ctypes

import pytest
import torch

from top_sparse_mla_gb300 import native
from top_sparse_mla_gb300.build import build

OK, BAD, SHAPE = native.DSA_OK, native.DSA_ERR_INVALID_ARG, native.DSA_ERR_UNSUPPORTED_SHAPE
NO_GPU = (native.DSA_ERR_CUDA, native.DSA_ERR_UNSUPPORTED_DEVICE)
FAKE = 1 << 20   # a 256-byte aligned address that is never dereferenced on the host


@pytest.fixture(scope="module")
def lib():
    build()
    return native.library()


def test_page_map(lib):
    args = dict(ctx=FAKE, new=FAKE, n=4, table=FAKE, ld=8, cols=8, free=FAKE, n_free=9, page=64, t=10, cu=FAKE, kv=FAKE,
                pos=FAKE, slots=FAKE, req=FAKE, info=FAKE)

    def call(**kw):
        a = dict(args, **kw)
        return lib.dsa_page_map(a["ctx"], a["new"], a["n"], a["table"], a["ld"], a["cols"], a["free"], a["n_free"],
                                a["page"], a["t"], a["cu"], a["kv"], a["pos"], a["slots"], a["req"], a["info"], None)

    for bad in (dict(n=-1), dict(t=-1), dict(t=(1 << 30) + 1), dict(page=0), dict(n_free=-1), dict(cols=0), dict(ld=7),
                dict(cols=1 << 29, ld=1 << 29), dict(ctx=None), dict(new=None), dict(table=None), dict(kv=None),
                dict(cu=None), dict(info=None), dict(free=None), dict(pos=None), dict(slots=None), dict(slots=FAKE + 4),
                dict(table=FAKE + 2), dict(req=FAKE + 1), dict(cu=FAKE + 2), dict(info=FAKE + 2)):
        assert call(**bad) == BAD, bad
    assert call(n=native.DSA_PAGE_MAP_MAX_REQ + 1) == SHAPE
    for ok in (dict(), dict(req=None), dict(t=0, pos=None, slots=None, req=None), dict(n_free=0, free=None),
               dict(n=0, ctx=None, new=None, table=None, kv=None, cols=0, ld=0)):
        assert call(**ok) in NO_GPU, ok


def test_insert(lib):
    args = dict(k=FAKE, k_ld=1024, k_hd=128, v=FAKE, v_ld=1024, v_hd=128, slots=FAKE, n=4, type=0, kp=FAKE, vp=FAKE,
                ks=FAKE, vs=FAKE, pages=10, h=8, page=64, d=128, status=None)

    def call(**kw):
        a = dict(args, **kw)
        return lib.dsa_kv8_insert(a["k"], a["k_ld"], a["k_hd"], a["v"], a["v_ld"], a["v_hd"], a["slots"], a["n"], a["type"],
                                  a["kp"], a["vp"], a["ks"], a["vs"], a["pages"], a["h"], a["page"], a["d"], a["status"], None)

    for bad in (dict(n=-1), dict(type=2), dict(pages=-1), dict(h=0), dict(k_ld=1028), dict(k_ld=120), dict(v_hd=64),
                dict(v_hd=132), dict(k=None), dict(v=None), dict(slots=None), dict(k=FAKE + 8), dict(v=FAKE + 2),
                dict(slots=FAKE + 4), dict(status=FAKE + 2), dict(kp=None), dict(vs=None), dict(kp=FAKE + 8),
                dict(ks=FAKE + 2)):
        assert call(**bad) == BAD, bad
    for shape in (dict(d=96), dict(d=256), dict(page=48), dict(page=256), dict(page=8), dict(h=1025), dict(pages=1 << 23)):
        assert call(**shape) == SHAPE, shape
    assert call(n=0, k=None, v=None, slots=None, kp=None) == OK      # an empty batch is a no-op
    for ok in (dict(), dict(h=1, k_hd=0, v_hd=0), dict(pages=0, kp=None, vp=None, ks=None, vs=None),
               dict(k_ld=128, k_hd=1 << 20)):                        # head-major keys
        assert call(**ok) in NO_GPU, ok


def _params(lib, **kw):
    p = native.DsaKv8Params()
    assert lib.dsa_kv8_params_init(ctypes.byref(p), 10, 4, 64, 8, 128, 64, 100, 16) == OK
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def test_attention(lib):
    p = _params(lib)
    assert (p.max_q_len, p.window, p.type, p.flags) == (10, 0, 0, 0) and abs(p.softmax_scale - 128 ** -0.5) < 1e-8
    size = lib.dsa_kv8_attn_workspace_size(ctypes.byref(p), 152)
    assert size > 0
    args = dict(q=FAKE, q_ld=8192, q_hd=128, kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE, table=FAKE, ld=16, cu=FAKE, kv=FAKE,
                out=FAKE, out_ld=8192, out_hd=128, lse=None, ws=FAKE, bytes=1 << 40)

    def call(p, **kw):
        a = dict(args, **kw)
        return lib.dsa_kv8_attn_fwd(a["q"], a["q_ld"], a["q_hd"], a["kp"], a["vp"], a["ks"], a["vs"], a["table"], a["ld"],
                                    a["cu"], a["kv"], a["out"], a["out_ld"], a["out_hd"], a["lse"],
                                    None if p is None else ctypes.byref(p), a["ws"], a["bytes"], None)

    assert call(None) == BAD
    for bad in (dict(n_tokens=-1), dict(n_req=-1), dict(h_q=60), dict(h_q=0), dict(h_kv=0), dict(n_pages=-1),
                dict(table_cols=-1), dict(max_q_len=-1), dict(window=-1), dict(type=2), dict(flags=1),
                dict(softmax_scale=float("nan")), dict(softmax_scale=float("inf"))):
        assert call(_params(lib, **bad)) == BAD, bad
        assert lib.dsa_kv8_attn_workspace_size(ctypes.byref(_params(lib, **bad)), 152) == 0
    for shape in (dict(d=96), dict(page_size=48), dict(n_req=8193), dict(h_kv=2048, h_q=2048), dict(h_q=129 * 8),
                  dict(n_tokens=1 << 30), dict(n_pages=1 << 23), dict(window=(1 << 30) + 1, table_cols=1 << 25)):
        assert call(_params(lib, **shape), ld=1 << 25) == SHAPE, shape
    assert call(_params(lib, window=(1 << 31) - 1)) in NO_GPU
    for bad in (dict(q=None), dict(out=None), dict(cu=None), dict(kv=None), dict(table=None), dict(kp=None), dict(vs=None),
                dict(q=FAKE + 8), dict(out=FAKE + 4), dict(kp=FAKE + 8), dict(q_ld=8196), dict(q_hd=64), dict(out_hd=132),
                dict(out_ld=64), dict(ld=15), dict(ws=None), dict(ws=FAKE + 16), dict(lse=FAKE + 2)):
        assert call(p, **bad) == BAD, bad
    # valid arguments reach the device check, which fails without a GPU
    assert call(p) in NO_GPU
    assert call(_params(lib, n_tokens=0), q=None, out=None) in NO_GPU
    assert call(_params(lib, n_pages=0, table_cols=0), kp=None, vp=None, ks=None, vs=None, table=None) in NO_GPU


def test_the_binding_refuses_tensors_that_do_not_fit(lib):
    i32 = torch.int32
    n, t = 3, 5
    ok = dict(ctx=torch.zeros(n, dtype=i32), new=torch.zeros(n, dtype=i32), table=torch.zeros((n, 4), dtype=i32),
              free=torch.zeros(2, dtype=i32), cu=torch.zeros(n + 1, dtype=i32), kv=torch.zeros(n, dtype=i32),
              pos=torch.zeros(t, dtype=i32), slots=torch.zeros(t, dtype=torch.int64), req=torch.zeros(t, dtype=i32),
              info=torch.zeros(2, dtype=i32))

    def page_map(**kw):
        a = dict(ok, **kw)
        native.dsa_page_map(a["ctx"], a["new"], a["table"], a["free"], 64, a["cu"], a["kv"], a["pos"], a["slots"], a["req"],
                            a["info"])

    for bad in (dict(), dict(new=torch.zeros(n + 1, dtype=i32)), dict(slots=torch.zeros(t, dtype=i32)),
                dict(pos=torch.zeros(2 * t, dtype=i32)[::2]), dict(cu=torch.zeros(n, dtype=i32)),
                dict(table=torch.zeros((4, n), dtype=i32).T)):
        with pytest.raises(native.DsaError) as e:   # the first: tensors that are not on a CUDA device
            page_map(**bad)
        assert e.value.code == BAD
    pool = torch.zeros((4, 2, 16, 64), dtype=torch.uint8)
    scale = torch.ones((4, 2))
    k = torch.zeros((t, 2, 64), dtype=torch.bfloat16)
    for kk, pp, ss in ((k, pool, scale), (k.float(), pool, scale), (k[:, :1], pool, scale), (k, pool[:, :, ::2], scale),
                       (k, pool, scale.double()), (k.transpose(0, 1), pool, scale)):
        with pytest.raises(native.DsaError) as e:
            native.dsa_kv8_insert(kk, kk, ok["slots"], pp, pp, ss, ss)
        assert e.value.code == BAD
    q, table = torch.zeros((t, 4, 64), dtype=torch.bfloat16), ok["table"]
    with pytest.raises(native.DsaError):
        native.dsa_kv8_params_init(q, pool, table, no_such_parameter=1)
    with pytest.raises(native.DsaError):
        native.dsa_kv8_params_init(q.float(), pool, table)
    p = native.dsa_kv8_params_init(q, pool, table, max_q_len=2, window=7)
    assert (p.n_tokens, p.n_req, p.h_q, p.h_kv, p.d, p.page_size, p.n_pages, p.table_cols, p.max_q_len, p.window) == (
        t, n, 4, 2, 64, 16, 4, 4, 2, 7)
    ws = torch.zeros(256, dtype=torch.uint8)
    for qq, out, tb in ((q, q.clone(), table), (q.half(), q.clone(), table), (q, q.clone().half(), table),
                        (q, q.clone()[:3], table), (q, q.clone(), table[:2])):
        with pytest.raises(native.DsaError) as e:
            native.dsa_kv8_attn_fwd(qq, pool, pool, scale, scale, tb, ok["cu"], ok["kv"], out, p, ws)
        assert e.value.code == BAD
