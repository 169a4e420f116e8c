"""The heads' norm, the cache read-back and the attentions beside the caches captured as a process's first calls, and called by several
host threads at once."""

import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from oracle import heads
from test_kv8_prefix_gpu import PrefixCase
from test_mla_prefill_gpu import Case as LatentCase
from top_sparse_mla_gb300 import native

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from top_sparse_mla_gb300.build import build
    build()
    native.library()


def _captured(call):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    return graph


def _latent(c, D, **kw):
    """A call's tensors and the call."""
    p = c.params(D, **kw)
    out = torch.full((c.n, c.h, 128), 7.0, dtype=c.q.dtype, device="cuda")
    lse = torch.full((c.n, c.h), 7.0, device="cuda")
    ws = torch.empty(native.dsa_mla_prefill_workspace_size(p), dtype=torch.uint8, device="cuda")
    return out, lse, lambda: native.dsa_mla_prefill_fwd(D["q"], D["k"], D["r"], D["v"], D["cu"], D["ck"], out, p, ws, lse=lse)


def _prefix(c, D):
    p = native.dsa_kv8_params_init(D["q"], D["kp"], D["table"], max_q_len=max(q for q, _ in c.lens), softmax_scale=c.scale)
    out = torch.full((c.n, c.h * c.g, c.d), 7.0, dtype=c.q.dtype, device="cuda")
    lse = torch.full((c.n, c.h * c.g), 7.0, device="cuda")
    ws = torch.empty(native.dsa_kv8_prefix_workspace_size(p, len(c.prefix)), dtype=torch.uint8, device="cuda")
    return out, lse, lambda: native.dsa_kv8_prefix_attn_fwd(D["q"], D["kp"], D["vp"], D["ks"], D["vs"], D["table"], D["cu"], D["kv"], D["cug"],
                                                            D["pre"], out, p, ws, lse=lse)


PREFIX = {"few": ([(1, 300)] * 4, [(4, 256)], 4), "shared out": ([(1, 700 + i) for i in range(40)], [(40, 688)], 8),
          "whole tiles": ([(40, 340)] * 60, [(60, 288)], 8), "many requests": ([(1, 60)] * 900, [(900, 48)], 4)}


def first_calls(which):
    """One operator's first call of the process is captured (no warm-up), replayed and checked."""
    if which == "norm":
        x = torch.randn((5, 3, 64), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
        q, pos = x.cuda(), torch.arange(5, dtype=torch.int32, device="cuda")
        out = torch.zeros_like(q)
        p = native.dsa_qk_params_init(q)
        _captured(lambda: native.dsa_qk_norm_rope(q, None, pos, None, None, out, None, p)).replay()
        want, _ = heads.norm_rope(x.double().numpy(), None, range(5), 64)
        assert np.abs(out.double().cpu().numpy() - want).max() <= 2.0 ** -8 * np.abs(want).max()
    elif which == "read-back":
        pool = torch.zeros((32, 656), dtype=torch.uint8, device="cuda")
        pool[:, :512], pool[:, 512:528] = 0x38, torch.tensor([2.0] * 4).view(torch.uint8).cuda()   # codes of 1, scales of 2
        out = torch.zeros((3, 576), dtype=torch.bfloat16, device="cuda")
        table, cu = torch.tensor([[1]], dtype=torch.int32, device="cuda"), torch.tensor([0, 3], dtype=torch.int32, device="cuda")
        _captured(lambda: native.dsa_kv_gather(pool, table, cu, out, 16)).replay()
        assert (out[:, :512] == 2).all() and (out[:, 512:] == 0).all()
    else:
        if which.startswith("latent"):
            c = LatentCase(31, [(70, 900), (300, 300)] if which == "latent split" else [(130, 200)] * 90, h=2 if which == "latent split" else 4)
            out, lse, call = _latent(c, c.device())
        else:
            lens, groups, g = PREFIX[which]
            c = PrefixCase(32, lens, groups, page=16, h=2, g=g, d=64)
            out, lse, call = _prefix(c, c.device())
        _captured(call).replay()
        torch.cuda.synchronize()
        c.check(out, lse)


@pytest.mark.parametrize("which", ["norm", "read-back", "latent split", "latent whole", *PREFIX])
def test_a_process_s_first_call_may_be_captured(which):
    code = f"import test_heads_capture_gpu as t; t.first_calls({which!r})"
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([here, os.path.dirname(here), os.environ.get("PYTHONPATH", "")]))
    run = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]


def test_several_host_threads_with_workspaces_of_their_own():
    cases = [LatentCase(41, [(70, 900)], h=4), LatentCase(42, [(130, 200)] * 60, h=4, dtype="fp16"),
             PrefixCase(43, *PREFIX["shared out"][:2], page=16, h=2, g=8, d=128), PrefixCase(44, *PREFIX["few"][:2], page=32, h=2, g=4, d=64)]
    made = [(_latent if isinstance(c, LatentCase) else _prefix)(c, c.device()) for c in cases]
    want = []
    for out, lse, call in made:
        call()
        torch.cuda.synchronize()
        want.append((out.clone(), lse.clone()))
    for c, (out, lse) in zip(cases, want):
        c.check(out, lse)
    failures = []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            out, lse, call = made[i]
            with torch.cuda.stream(stream):
                for _ in range(40):
                    out.fill_(7.0)
                    call()
                    stream.synchronize()
                    if not (torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])):
                        failures.append((i, "another result"))
        except Exception as e:   # noqa: BLE001
            failures.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures[:3]


def test_two_graphs_in_turn_with_one_workspace():
    """Calls that share a workspace may follow one another, captured or not."""
    a, b = PrefixCase(51, *PREFIX["shared out"][:2], page=16, h=2, g=8, d=64), PrefixCase(52, [(1, 500 + i) for i in range(40)], [(40, 496)], page=16,
                                                                                          h=2, g=8, d=64)
    Da, Db = a.device(), b.device()
    ps = [native.dsa_kv8_params_init(D["q"], D["kp"], D["table"], max_q_len=1, softmax_scale=c.scale) for c, D in ((a, Da), (b, Db))]
    ws = torch.empty(max(native.dsa_kv8_prefix_workspace_size(p, 1) for p in ps), dtype=torch.uint8, device="cuda")
    outs = [(torch.full((c.n, 16, 64), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((c.n, 16), 7.0, device="cuda")) for c in (a, b)]

    def call(c, D, p, out, lse):
        native.dsa_kv8_prefix_attn_fwd(D["q"], D["kp"], D["vp"], D["ks"], D["vs"], D["table"], D["cu"], D["kv"], D["cug"], D["pre"], out, p, ws, lse=lse)

    graphs = [_captured(lambda c=c, D=D, p=p, o=o: call(c, D, p, *o)) for c, D, p, o in zip((a, b), (Da, Db), ps, outs)]
    for _ in range(3):
        for out, lse in outs:
            out.fill_(7.0)
            lse.fill_(7.0)
        for g in graphs:
            g.replay()
        call(a, Da, ps[0], *outs[0])
        torch.cuda.synchronize()
        for c, (out, lse) in zip((a, b), outs):
            c.check(out, lse)
