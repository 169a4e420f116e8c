"""Host-side checks of the entry points that make heads ready and of the attentions beside the caches (no GPU): arguments are
refused by the C ABI before anything touches a GPU."""

import ctypes

import pytest

from top_sparse_mla_gb300 import native
from top_sparse_mla_gb300.build import build

OK, BAD, SHAPE, SMALL = native.DSA_OK, native.DSA_ERR_INVALID_ARG, native.DSA_ERR_UNSUPPORTED_SHAPE, native.DSA_ERR_WORKSPACE_TOO_SMALL
NO_GPU = (native.DSA_ERR_CUDA, native.DSA_ERR_UNSUPPORTED_DEVICE)
FAKE = 1 << 20   # a 256-byte aligned address that is never dereferenced on the host
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    build()
    return native.library()


def _set(p, kw):
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def test_norm_rope(lib):
    def params(**kw):
        p = native.DsaQkParams()
        assert lib.dsa_qk_params_init(ctypes.byref(p), 10, 8, 2, 128) == OK
        return _set(p, kw)

    p = params()
    assert (p.rotary_dim, p.rotary_start, p.type, p.flags, p.rope_base) == (128, 0, 0, 0, 10000.0) and abs(p.rms_eps - 1e-6) < 1e-12
    args = dict(q=FAKE, q_ld=1024, q_hd=128, k=FAKE, k_ld=256, k_hd=128, pos=FAKE, qw=FAKE, kw=FAKE, qo=2 * FAKE, qo_ld=1024, qo_hd=128,
                ko=3 * FAKE, ko_ld=256, ko_hd=128)

    def call(p, **kw):
        a = dict(args, **kw)
        return lib.dsa_qk_norm_rope(a["q"], a["q_ld"], a["q_hd"], a["k"], a["k_ld"], a["k_hd"], a["pos"], a["qw"], a["kw"], a["qo"],
                                    a["qo_ld"], a["qo_hd"], a["ko"], a["ko_ld"], a["ko_hd"], None if p is None else ctypes.byref(p), None)

    assert call(None) == BAD and lib.dsa_qk_params_init(None, 1, 1, 1, 64) == BAD
    for bad in (dict(n_tokens=-1), dict(n_tokens=(1 << 30) + 1), dict(h_q=0), dict(h_k=-1), dict(rotary_dim=-16), dict(rotary_start=-8),
                dict(type=2), dict(flags=2), dict(rms_eps=-1.0), dict(rms_eps=NAN), dict(rms_eps=INF), dict(rope_base=0.0),
                dict(rope_base=-1.0), dict(rope_base=NAN), dict(rope_base=INF)):
        assert call(params(**bad)) == BAD, bad
    for shape in (dict(d=48), dict(d=72), dict(d=272), dict(rotary_dim=136), dict(rotary_dim=24), dict(rotary_dim=64, rotary_start=72),
                  dict(rotary_dim=64, rotary_start=4), dict(h_q=4097), dict(h_q=4000, h_k=97)):
        assert call(params(**shape)) == SHAPE, shape
    for bad in (dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(pos=None), dict(q=FAKE + 8), dict(ko=FAKE + 2), dict(qw=FAKE + 8),
                dict(kw=FAKE + 4), dict(pos=FAKE + 2), dict(q_ld=1028), dict(q_ld=120), dict(k_hd=64), dict(qo_hd=132), dict(ko_ld=-128),
                dict(qo=FAKE, qo_ld=2048), dict(ko=FAKE, ko_hd=256)):
        assert call(p, **bad) == BAD, bad
    assert call(params(n_tokens=0), q=None, k=None, pos=None, qo=None, ko=None) == OK
    for ok in (dict(), dict(qw=None), dict(kw=None), dict(qo=FAKE), dict(q_ld=1 << 20, q_hd=1 << 30)):
        assert call(p, **ok) in NO_GPU, ok
    assert call(params(h_k=0), k=None, ko=None, kw=None, k_ld=3) in NO_GPU
    assert call(params(rotary_dim=0)) in NO_GPU and call(params(n_tokens=1), q_ld=8) in NO_GPU


def test_gather(lib):
    args = dict(pool=FAKE, rows=100, table=FAKE, ld=8, cols=8, page=64, cu=FAKE, lens=None, n=4, out=FAKE, out_ld=576, n_out=10, status=None)

    def call(**kw):
        a = dict(args, **kw)
        return lib.dsa_kv_gather(a["pool"], a["rows"], a["table"], a["ld"], a["cols"], a["page"], a["cu"], a["lens"], a["n"], a["out"],
                                 a["out_ld"], a["n_out"], a["status"], None)

    for bad in (dict(rows=-1), dict(n=-1), dict(n_out=-1), dict(cols=-1), dict(page=0), dict(out_ld=568), dict(out_ld=580), dict(status=FAKE + 2),
                dict(cu=None), dict(out=None), dict(pool=None), dict(table=None), dict(cu=FAKE + 2), dict(out=FAKE + 8), dict(lens=FAKE + 1),
                dict(pool=FAKE + 8), dict(table=FAKE + 2), dict(ld=7)):
        assert call(**bad) == BAD, bad
    assert call(n=0, cu=None, out=None) == OK and call(n_out=0, out=None) == OK
    for ok in (dict(), dict(rows=0, pool=None), dict(cols=0, table=None), dict(n=1, ld=0), dict(lens=FAKE, status=FAKE + 4), dict(page=1)):
        assert call(**ok) in NO_GPU, ok


def test_latent_attention(lib):
    def params(**kw):
        p = native.DsaMlaParams()
        assert lib.dsa_mla_params_init(ctypes.byref(p), 10, 50, 4, 16) == OK
        return _set(p, kw)

    p = params()
    assert (p.max_q_len, p.max_kv_len, p.type, p.flags) == (10, 50, 0, 0) and abs(p.softmax_scale - 192 ** -0.5) < 1e-8
    size = lib.dsa_mla_prefill_workspace_size(ctypes.byref(p), 152)
    assert size > 0
    args = dict(q=FAKE, q_ld=3200, q_hd=200, k=FAKE, k_ld=4096, k_hd=256, r=FAKE, r_ld=576, v=FAKE, v_ld=4096, v_hd=256, cu=FAKE, ck=FAKE,
                out=FAKE, out_ld=2048, out_hd=128, lse=None, ws=FAKE, bytes=1 << 40)

    def call(p, **kw):
        a = dict(args, **kw)
        return lib.dsa_mla_prefill_fwd(a["q"], a["q_ld"], a["q_hd"], a["k"], a["k_ld"], a["k_hd"], a["r"], a["r_ld"], a["v"], a["v_ld"],
                                       a["v_hd"], a["cu"], a["ck"], a["out"], a["out_ld"], a["out_hd"], a["lse"],
                                       None if p is None else ctypes.byref(p), a["ws"], a["bytes"], None)

    assert call(None) == BAD and lib.dsa_mla_params_init(None, 1, 1, 1, 1) == BAD
    assert lib.dsa_mla_prefill_workspace_size(None, 152) == 0
    for bad in (dict(n_tokens=-1), dict(n_keys=-1), dict(n_req=-1), dict(h=0), dict(max_q_len=-1), dict(max_kv_len=-1), dict(type=2), dict(flags=1),
                dict(softmax_scale=NAN), dict(softmax_scale=INF)):
        assert call(params(**bad)) == BAD, bad
        assert lib.dsa_mla_prefill_workspace_size(ctypes.byref(params(**bad)), 152) == 0
    for shape in (dict(n_req=8193), dict(h=1025), dict(n_tokens=(1 << 30) + 1), dict(n_keys=(1 << 30) + 1)):
        assert call(params(**shape)) == SHAPE, shape
    for bad in (dict(q=None), dict(k=None), dict(r=None), dict(v=None), dict(out=None), dict(cu=None), dict(ck=None), dict(ws=None),
                dict(ws=FAKE + 16), dict(q=FAKE + 8), dict(r=FAKE + 8), dict(v=FAKE + 2), dict(out=FAKE + 4), dict(cu=FAKE + 2), dict(ck=FAKE + 1),
                dict(lse=FAKE + 2), dict(q_ld=3204), dict(q_hd=184), dict(k_hd=0), dict(k_ld=64), dict(r_ld=60), dict(r_ld=56), dict(v_hd=132),
                dict(v_ld=-4096), dict(out_hd=120), dict(q_ld=1 << 37), dict(r_ld=1 << 37)):
        assert call(p, **bad) == BAD, bad
    assert call(p) in NO_GPU
    assert call(params(n_tokens=0), q=None, out=None) in NO_GPU and call(params(n_keys=0), k=None, r=None, v=None) in NO_GPU
    assert call(params(h=1), q_hd=0, k_hd=0, v_hd=0, out_hd=0) in NO_GPU


def test_prefix_attention(lib):
    def params(**kw):
        p = native.DsaKv8Params()
        assert lib.dsa_kv8_params_init(ctypes.byref(p), 10, 4, 64, 8, 128, 64, 100, 16) == OK
        return _set(p, kw)

    p = params()
    assert lib.dsa_kv8_prefix_workspace_size(ctypes.byref(p), 2, 152) > 0
    args = dict(q=FAKE, q_ld=8192, q_hd=128, kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE, table=FAKE, ld=16, cu=FAKE, kv=FAKE, cg=FAKE, pl=FAKE, groups=2,
                out=FAKE, out_ld=8192, out_hd=128, lse=None, ws=FAKE, bytes=1 << 40)

    def call(p, **kw):
        a = dict(args, **kw)
        return lib.dsa_kv8_prefix_attn_fwd(a["q"], a["q_ld"], a["q_hd"], a["kp"], a["vp"], a["ks"], a["vs"], a["table"], a["ld"], a["cu"],
                                           a["kv"], a["cg"], a["pl"], a["groups"], a["out"], a["out_ld"], a["out_hd"], a["lse"],
                                           None if p is None else ctypes.byref(p), a["ws"], a["bytes"], None)

    assert call(None) == BAD
    for bad in (dict(n_tokens=-1), dict(h_q=60), dict(window=-1), dict(type=2), dict(flags=1), dict(softmax_scale=NAN)):
        assert call(params(**bad)) == BAD, bad
        assert lib.dsa_kv8_prefix_workspace_size(ctypes.byref(params(**bad)), 2, 152) == 0
    for shape in (dict(d=96), dict(page_size=48), dict(n_req=8193), dict(window=1)):
        assert call(params(**shape)) == SHAPE, shape
    assert call(p, groups=-1) == BAD and call(p, groups=native.DSA_KV8_MAX_GROUPS + 1) == SHAPE
    assert call(params(n_req=8191), groups=2) == SHAPE and call(params(n_req=8190), groups=2) in NO_GPU
    for bad in (dict(q=None), dict(out=None), dict(cu=None), dict(kv=None), dict(table=None), dict(kp=None), dict(vs=None), dict(cg=None),
                dict(pl=None), dict(cg=FAKE + 2), dict(pl=FAKE + 1), dict(q=FAKE + 8), dict(q_hd=64), dict(ld=15), dict(ws=None),
                dict(ws=FAKE + 16), dict(lse=FAKE + 2)):
        assert call(p, **bad) == BAD, bad
    assert call(p) in NO_GPU and call(p, groups=0, cg=None, pl=None) in NO_GPU
    assert call(params(n_tokens=0), q=None, out=None) in NO_GPU
