"""Cases of the operators that make a layer's queries and keys ready and of the two attentions beside the caches: the
heads' norm and rotation (dsa_qk_norm_rope), latent rows read back from the cache (dsa_kv_gather), latent attention with
expanded keys and values (dsa_mla_prefill_fwd), and attention over the paged 8-bit cache for requests that share a prefix
(dsa_kv8_prefix_attn_fwd).

`run` computes them in elementary torch operations, or, where `own` is true, with the library's entry points; `exact`
restates each definition in 64 bits.

Definitions.
  qk      y = x / sqrt(mean(x^2) + eps) * w over a head's d values (y = x without weights); the rotary pairs of y, (i, i + rot / 2)
          or, interleaved, (2i, 2i + 1), counted from `start`, are rotated by position * base^(-2i / rot).
  gather  row cu[r] + i of out = row i of request r in the cache: page table[r][i / P], 512 E4M3 codes times one fp32 scale
          for each 128 of them, then 64 bf16 values as they are.
  mla     query i of request r sees the keys j <= kv_len - q_len + i of its request; a key of head h is (k_nope[j][h], k_rope[j]),
          192 dims; out = softmax(scale * q.k) v, lse = the natural-log sum-exp.
  prefix  query i of request r is at position kv_len[r] - q_len[r] + i and sees the cached tokens j <= its own position; the
          requests of a group have the same pages for their first prefix_len tokens (whole pages of them)."""

import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # a decode step's heads, out of a packed qkv projection: latency alone
        {"name": "qk_decode_64", "op": "qk", "n": 64, "h_q": 64, "h_k": 8, "d": 128, "rot": 128, "start": 0, "inter": False, "norm": True,
         "dtype": "bf16", "pos_max": 32768},
        # a prefill wave: memory bound
        {"name": "qk_prefill_16381", "op": "qk", "n": 16381, "h_q": 64, "h_k": 8, "d": 128, "rot": 128, "start": 0, "inter": False,
         "norm": True, "dtype": "bf16", "pos_max": 131072},
        # a latent layer's queries: only the last 64 dims turn, no norm, fp16
        {"name": "qk_latent_2123", "op": "qk", "n": 2123, "h_q": 16, "h_k": 0, "d": 192, "rot": 64, "start": 128, "inter": True,
         "norm": False, "dtype": "fp16", "pos_max": 8192},
        # one request's short context in front of its next chunk
        {"name": "gather_1", "op": "gather", "n_req": 1, "ctx_max": 1000, "page": 64, "lens": 1},
        # the contexts of a wave of chunks
        {"name": "gather_24", "op": "gather", "n_req": 24, "ctx_max": 8192, "page": 16, "lens": 2},
        # many short prompts at once, a tensor-parallel share of the heads, fp16
        {"name": "mla_short_64", "op": "mla", "n_req": 64, "q_max": 128, "kv_max": 128, "h": 8, "dtype": "fp16", "lens": 3},
        # one prompt of an odd length from its start
        {"name": "mla_prefill_2123", "op": "mla", "n_req": 1, "q_max": 2123, "kv_max": 2123, "h": 64, "dtype": "bf16", "lens": 4},
        # few new tokens behind a long context: split along the keys
        {"name": "mla_tail_64_on_32k", "op": "mla", "n_req": 1, "q_max": 64, "kv_max": 32768, "h": 16, "dtype": "bf16", "lens": 5},
        # ragged chunks of several requests behind contexts of their own
        {"name": "mla_chunks_6", "op": "mla", "n_req": 6, "q_max": 2048, "kv_max": 8192, "h": 32, "dtype": "bf16", "lens": 6},
        # a few answers sampled from one short prompt
        {"name": "prefix_decode_4", "op": "prefix", "groups": 1, "n_req": 4, "q_max": 1, "prefix_max": 2048, "own_max": 128, "h_q": 32, "h": 8,
         "d": 128, "page": 64, "dtype": "bf16", "lens": 7},
        # a batch behind one long system prompt
        {"name": "prefix_decode_64", "op": "prefix", "groups": 1, "n_req": 64, "q_max": 1, "prefix_max": 16391, "own_max": 1024, "h_q": 64,
         "h": 8, "d": 128, "page": 64, "dtype": "bf16", "lens": 8},
        # several prompts, many samples of each, drafted tokens verified at once, a small model
        {"name": "prefix_verify_240", "op": "prefix", "groups": 5, "n_req": 240, "q_max": 4, "prefix_max": 4096, "own_max": 512, "h_q": 16,
         "h": 2, "d": 64, "page": 16, "dtype": "fp16", "lens": 9},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qk", "gather", "mla", "mla", "prefix", "prefix"])
    dtype = rng.choice(["bf16", "fp16"])
    lens = rng.randrange(1, 1 << 20)
    if op == "qk":
        d = rng.choice([64, 128, 128, 192, 256])
        inter = rng.random() < 0.4
        rot = rng.choice([d, d // 2, 64])
        h_k = rng.choice([0, 1, 2, 4, 8])
        h_q = max(1, h_k) * rng.choice([1, 4, 5, 8])
        n = _log_int(rng, 1, min(32768, (1 << 27) // ((h_q + h_k) * d)))
        return {"op": op, "n": n, "h_q": h_q, "h_k": h_k, "d": d, "rot": rot, "start": rng.choice([0, d - rot]), "inter": inter,
                "norm": rng.random() < 0.7, "dtype": dtype, "pos_max": _log_int(rng, 128, 1 << 20)}
    if op == "gather":
        n_req = _log_int(rng, 1, 256)
        return {"op": op, "n_req": n_req, "ctx_max": _log_int(rng, 1, min(32768, 160000 // n_req)), "page": rng.choice([16, 32, 64, 128]),
                "lens": lens}
    if op == "mla":
        h = rng.choice([1, 4, 8, 16, 32])
        if rng.random() < 0.3:   # many short ones
            n_req = _log_int(rng, 8, 128)
            kv_max = _log_int(rng, 1, 512)
        else:
            n_req = rng.choice([1, 2, 3, 5])
            kv_max = _log_int(rng, 64, 8192)
        return {"op": op, "n_req": n_req, "q_max": _log_int(rng, 1, min(kv_max, 4096)), "kv_max": kv_max, "h": h, "dtype": dtype, "lens": lens}
    groups = rng.choice([1, 1, 2, 5])
    n_req = max(groups, _log_int(rng, 1, 384))
    prefix_max = _log_int(rng, 16, min(32768, (1 << 20) // n_req))
    h = rng.choice([1, 2, 4, 8])
    return {"op": op, "groups": groups, "n_req": n_req, "q_max": rng.choice([1, 1, 2, 4]), "prefix_max": prefix_max,
            "own_max": _log_int(rng, 4, 1024), "h_q": h * rng.choice([1, 4, 8]), "h": h, "d": rng.choice([64, 128]),
            "page": rng.choice([16, 32, 64, 128]), "dtype": dtype, "lens": lens}


# ------------------------------------------------------------------------------ sizes
def _lens(case):
    """Lengths of a case.  They belong to the case, not to the seed.  gather: (context lengths, None); mla: (key counts, query
    counts); prefix: (lengths, query counts, requests of each group, prefix lengths)."""
    r = random.Random(case["lens"])
    n = case["n_req"]
    if case["op"] == "gather":
        ctx = [r.randint(0, case["ctx_max"]) for _ in range(n)]
        ctx[0] = case["ctx_max"]
        return ctx, None
    if case["op"] == "mla":
        q = [r.randint(max(1, case["q_max"] // 2), case["q_max"]) for _ in range(n)]
        kv = [r.randint(a, case["kv_max"]) for a in q]
        q[0], kv[0] = case["q_max"], case["kv_max"]
        return kv, q
    g = case["groups"]
    size = [n // g + (1 if i < n % g else 0) for i in range(g)]
    pre = [r.randint(max(1, case["prefix_max"] // 2), case["prefix_max"]) for _ in range(g)]
    pre[0] = case["prefix_max"]
    q = [r.randint(1, case["q_max"]) for _ in range(n)]
    group = [i for i in range(g) for _ in range(size[i])]
    kv = [pre[group[i]] + q[i] + r.randint(0, max(0, case["own_max"] - q[i])) for i in range(n)]
    return kv, q, size, pre


def _cdiv(a, b):
    return -(-a // b)


def _prefix(v):
    return [0] + list(np.cumsum(np.asarray(v, dtype=np.int64)).tolist())


def _pairs(kv, q):
    """Visible (query, key) pairs of one request."""
    return q * kv - q * (q - 1) // 2


def work(case):
    if case["op"] == "qk":
        values = case["n"] * (case["h_q"] + case["h_k"]) * case["d"]
        return {"bytes": 4 * values + 4 * case["n"] + (4 * case["d"] if case["norm"] else 0), "flops": 8 * values}
    if case["op"] == "gather":
        rows = sum(_lens(case)[0])
        return {"bytes": rows * (656 + 1152), "flops": 512 * rows}
    if case["op"] == "mla":
        kv, q = _lens(case)
        h = case["h"]
        return {"bytes": sum(q) * h * (2 * 192 + 2 * 128 + 4) + sum(kv) * (h * 512 + 128),
                "flops": 2 * sum(_pairs(a, b) for a, b in zip(kv, q)) * h * (192 + 128)}
    kv, q, size, pre = _lens(case)
    page, h, d = case["page"], case["h"], case["d"]
    shared = [p // page * page for p in pre]
    group = [i for i in range(len(size)) for _ in range(size[i])]
    cached = sum(shared) + sum(a - shared[g] for a, g in zip(kv, group))
    return {"bytes": cached * h * d * 2 + sum(q) * case["h_q"] * (4 * d + 4) + _cdiv(cached, page) * (4 + 8 * h),
            "flops": 4 * sum(_pairs(a, b) for a, b in zip(kv, q)) * case["h_q"] * d}


# ------------------------------------------------------------------------------ inputs
def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _randn(shape, gen, dtype):
    """Normal values of a 16-bit type, some million at a time."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for a in range(0, flat.numel(), 1 << 26):
        b = min(a + (1 << 26), flat.numel())
        flat[a:b] = torch.randn(b - a, generator=gen, device="cuda")
    return out


def _prepare_qk(case, gen):
    n, h_q, h_k, d, dtype = case["n"], case["h_q"], case["h_k"], case["d"], DTYPES[case["dtype"]]
    # queries and keys inside a packed qkv projection's output
    qkv = _randn((n, h_q + 2 * h_k, d), gen, dtype)
    qkv[:, :, ::19] *= 5.0   # a few channels carry most of the magnitude
    st = {"op": "qk", "rot": case["rot"], "start": case["start"], "inter": case["inter"], "eps": 1e-6, "base": 10000.0,
          "q": qkv[:, :h_q], "k": qkv[:, h_q:h_q + h_k] if h_k else None, "q_w": None, "k_w": None,
          "pos": torch.randint(0, case["pos_max"], (n,), generator=gen, device="cuda").to(torch.int32),
          "q_out": torch.empty((n, h_q, d), dtype=dtype, device="cuda"),
          "k_out": torch.empty((n, h_k, d), dtype=dtype, device="cuda") if h_k else None}
    if case["norm"]:
        st["q_w"] = (1.0 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(dtype)
        st["k_w"] = (1.0 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(dtype) if h_k else None
    if own:
        from top_sparse_mla_gb300 import native
        st["params"] = native.dsa_qk_params_init(st["q"], st["k"], rotary_dim=st["rot"], rotary_start=st["start"],
                                                 interleaved=st["inter"], rms_eps=st["eps"], rope_base=st["base"])
    return st


def _prepare_gather(case, gen):
    ctx, _ = _lens(case)
    page, n = case["page"], case["n_req"]
    pages = [_cdiv(c, page) for c in ctx]
    cols, n_pages = max(max(pages), 1), sum(pages) + 3
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    start = _ints(_prefix(pages)[:-1], torch.int64)
    col = torch.arange(cols, device="cuda")
    at = (start[:, None] + col[None, :]).clamp_(max=n_pages - 1)
    table = torch.where(col[None, :] < _ints(pages)[:, None], order[at], torch.full_like(order[at], -1)).contiguous()
    rows = n_pages * page
    pool = torch.empty((rows, 656), dtype=torch.uint8, device="cuda")
    # as the insert leaves a row: a block's largest code is 448, its scale the block's largest value over that
    x = torch.randn((rows, 4, 128), generator=gen, device="cuda")
    s = x.abs().amax(dim=2, keepdim=True) / 448.0
    pool[:, :512] = (x / s).reshape(rows, 512).to(torch.float8_e4m3fn).view(torch.uint8)
    pool[:, 512:528] = s.reshape(rows, 4).contiguous().view(torch.uint8)
    pool[:, 528:] = torch.randn((rows, 64), generator=gen, device="cuda").to(torch.bfloat16).view(torch.uint8)
    return {"op": "gather", "page": page, "pool": pool, "table": table, "cu": _ints(_prefix(ctx)),
            "out": torch.zeros((sum(ctx), 576), dtype=torch.bfloat16, device="cuda")}


def _prepare_mla(case, gen):
    kv, q = _lens(case)
    h, dtype = case["h"], DTYPES[case["dtype"]]
    t, s = sum(q), sum(kv)
    # keys and values side by side, as the up-projection of the latent rows leaves them; the rotary keys inside those rows
    up = _randn((s, h, 256), gen, dtype)
    latent = _randn((s, 576), gen, dtype)
    qs = _randn((t, h, 192), gen, dtype).mul_(1.5)
    st = {"op": "mla", "q": qs, "k_nope": up[:, :, :128], "v": up[:, :, 128:], "k_rope": latent[:, 512:], "cu_q": _ints(_prefix(q)),
          "cu_kv": _ints(_prefix(kv)), "q_lens": q, "kv_lens": kv, "scale": 1.0 / math.sqrt(192.0),
          "out": torch.empty((t, h, 128), dtype=dtype, device="cuda"), "lse": torch.empty((t, h), dtype=torch.float32, device="cuda")}
    if own:
        from top_sparse_mla_gb300 import native
        st["params"] = native.dsa_mla_params_init(qs, st["k_nope"], st["cu_q"], max_q_len=max(q), max_kv_len=max(kv))
        st["workspace"] = torch.empty(native.dsa_mla_prefill_workspace_size(st["params"]), dtype=torch.uint8, device="cuda")
    return st


def _cache(n_pages, h, page, d, gen):
    """A pool as the insert leaves it: a magnitude of its own for each page and head, and the power-of-two scale of that page."""
    pool = torch.empty((n_pages, h, page, d), dtype=torch.uint8, device="cuda")
    mag = torch.exp2(torch.randint(-2, 2, (n_pages, h), generator=gen, device="cuda").float())
    step = max(1, (1 << 26) // (h * page * d))
    for a in range(0, n_pages, step):
        x = torch.randn((min(step, n_pages - a), h, page, d), generator=gen, device="cuda")
        pool[a:a + step] = (x * 64.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return pool, (mag / 64.0).contiguous()


def _prepare_prefix(case, gen):
    kv, q, size, pre = _lens(case)
    n, page, h, d, dtype = case["n_req"], case["page"], case["h"], case["d"], DTYPES[case["dtype"]]
    shared = [p // page for p in pre]
    group = [i for i in range(len(size)) for _ in range(size[i])]
    used = [_cdiv(a, page) for a in kv]
    n_pages = sum(shared) + sum(u - shared[g] for u, g in zip(used, group)) + 3
    order = torch.randperm(n_pages, generator=gen, device="cuda").cpu().numpy().astype(np.int32)
    table = np.full((n, max(used)), -1, np.int32)
    at = sum(shared)
    first = _prefix(shared)
    for r, (u, g) in enumerate(zip(used, group)):
        table[r, :shared[g]] = order[first[g]:first[g] + shared[g]]
        table[r, shared[g]:u] = order[at:at + u - shared[g]]
        at += u - shared[g]
    k_pool, k_scale = _cache(n_pages, h, page, d, gen)
    v_pool, v_scale = _cache(n_pages, h, page, d, gen)
    t = sum(q)
    st = {"op": "prefix", "page": page, "k_pool": k_pool, "v_pool": v_pool, "k_scale": k_scale, "v_scale": v_scale,
          "q": _randn((t, case["h_q"], d), gen, dtype).mul_(2.0), "table": torch.from_numpy(table).cuda(), "cu": _ints(_prefix(q)),
          "kv_lens": _ints(kv), "cu_groups": _ints(_prefix(size)), "prefix_lens": _ints(pre), "q_max": max(q), "scale": 1.0 / math.sqrt(d),
          "out": torch.empty((t, case["h_q"], d), dtype=dtype, device="cuda"),
          "lse": torch.empty((t, case["h_q"]), dtype=torch.float32, device="cuda")}
    if own:
        from top_sparse_mla_gb300 import native
        st["params"] = native.dsa_kv8_params_init(st["q"], k_pool, st["table"], max_q_len=st["q_max"])
        size = native.dsa_kv8_prefix_workspace_size(st["params"], len(pre))
        st["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) & 0x7FFFFFFF)
    return {"qk": _prepare_qk, "gather": _prepare_gather, "mla": _prepare_mla, "prefix": _prepare_prefix}[case["op"]](case, gen)


# ------------------------------------------------------------------------------ plain forms
def _plain_qk_one(x, w, s):
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt(y.square().mean(dim=-1, keepdim=True) + s["eps"]) * w.float()
    else:
        y = y.clone()
    half = s["rot"] // 2
    i = torch.arange(half, device="cuda", dtype=torch.float64)
    angle = s["pos"].double()[:, None] * torch.exp(i * (-2.0 * math.log(s["base"]) / s["rot"]))[None, :]
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    a = s["start"]
    if s["inter"]:
        u, v = y[..., a:a + s["rot"]:2], y[..., a + 1:a + s["rot"]:2]
    else:
        u, v = y[..., a:a + half], y[..., a + half:a + s["rot"]]
    turned = u * cos - v * sin, u * sin + v * cos
    u.copy_(turned[0])
    v.copy_(turned[1])
    return y


def _plain_gather(s):
    cu, page = s["cu"].long(), s["page"]
    t = torch.arange(s["out"].shape[0], device="cuda")
    r = torch.searchsorted(cu[1:], t, right=True)
    i = t - cu[r]
    rows = s["pool"][s["table"][r, i // page].long() * page + i % page]
    codes = rows[:, :512].contiguous().view(torch.float8_e4m3fn).float().view(-1, 4, 128)
    scale = rows[:, 512:528].contiguous().view(torch.float32)
    s["out"][:, :512] = (codes * scale[:, :, None]).view(-1, 512)
    s["out"][:, 512:] = rows[:, 528:].contiguous().view(torch.bfloat16)


def _plain_mla(s):
    cu, ck = _prefix(s["q_lens"]), _prefix(s["kv_lens"])
    for r, (n, m) in enumerate(zip(s["q_lens"], s["kv_lens"])):
        q = s["q"][cu[r]:cu[r + 1]].float().transpose(0, 1)
        k = s["k_nope"][ck[r]:ck[r + 1]].float().transpose(0, 1)
        v = s["v"][ck[r]:ck[r + 1]].float().transpose(0, 1)
        x = torch.matmul(q[..., :128], k.transpose(1, 2))
        x += torch.matmul(q[..., 128:], s["k_rope"][ck[r]:ck[r + 1]].float().t())
        x *= s["scale"]
        i = torch.arange(m - n, m, device="cuda")[:, None]
        x.masked_fill_(torch.arange(m, device="cuda")[None, :] > i, float("-inf"))
        top = x.amax(dim=-1, keepdim=True)
        x = x.sub_(top).exp_()
        total = x.sum(dim=-1, keepdim=True)
        s["out"][cu[r]:cu[r + 1]] = (torch.matmul(x, v) / total).transpose(0, 1)
        s["lse"][cu[r]:cu[r + 1]] = (top + total.log())[..., 0].t()


def _plain_prefix(s):
    q, table, cu, kv = s["q"], s["table"].long().clamp(min=0), s["cu"].long(), s["kv_lens"].long()
    b, h_q, d = table.shape[0], q.shape[1], q.shape[2]
    h = s["k_pool"].shape[1]
    g, qm = h_q // h, s["q_max"]
    n = cu[1:] - cu[:-1]

    def rows(pool, scale):
        x = pool[table].view(torch.float8_e4m3fn).float() * scale[table][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(b, h, -1, d)

    k, v = rows(s["k_pool"], s["k_scale"]), rows(s["v_pool"], s["v_scale"])
    i = torch.arange(qm, device="cuda")
    at = (cu[:-1, None] + i[None, :]).clamp(max=q.shape[0] - 1)
    qp = q[at].float().reshape(b, qm, h, g, d).permute(0, 2, 1, 3, 4).reshape(b, h, qm * g, d)
    x = torch.matmul(qp, k.transpose(2, 3)).mul_(s["scale"])
    pos = (kv - n)[:, None] + i[None, :]
    seen = torch.arange(k.shape[2], device="cuda")[None, None, :] <= pos[:, :, None]
    x = x.view(b, h, qm, g, -1).masked_fill_(~seen[:, None, :, None, :], float("-inf")).view(b, h, qm * g, -1)
    top = x.amax(dim=-1, keepdim=True)
    x = x.sub_(top).exp_()
    total = x.sum(dim=-1, keepdim=True)
    o = (torch.matmul(x, v) / total).view(b, h, qm, g, d).permute(0, 2, 1, 3, 4).reshape(b, qm, h_q, d)
    lse = (top + total.log()).view(b, h, qm, g).permute(0, 2, 1, 3).reshape(b, qm, h_q)
    t = torch.arange(q.shape[0], device="cuda")
    r = torch.searchsorted(cu[1:], t, right=True)
    s["out"].copy_(o[r, t - cu[r]])
    s["lse"].copy_(lse[r, t - cu[r]])


def run(state):
    s = state
    if own:
        from top_sparse_mla_gb300 import native
    if s["op"] == "qk":
        if own:
            native.dsa_qk_norm_rope(s["q"], s["k"], s["pos"], s["q_w"], s["k_w"], s["q_out"], s["k_out"], s["params"])
        else:
            s["q_out"].copy_(_plain_qk_one(s["q"], s["q_w"], s))
            if s["k"] is not None:
                s["k_out"].copy_(_plain_qk_one(s["k"], s["k_w"], s))
        return {"q": s["q_out"], "k": s["k_out"]} if s["k"] is not None else {"q": s["q_out"]}
    if s["op"] == "gather":
        if own:
            native.dsa_kv_gather(s["pool"], s["table"], s["cu"], s["out"], s["page"])
        else:
            _plain_gather(s)
        return {"out": s["out"]}
    if s["op"] == "mla":
        if own:
            native.dsa_mla_prefill_fwd(s["q"], s["k_nope"], s["k_rope"], s["v"], s["cu_q"], s["cu_kv"], s["out"], s["params"],
                                       s["workspace"], lse=s["lse"])
        else:
            _plain_mla(s)
        return {"out": s["out"], "lse": s["lse"]}
    if own:
        native.dsa_kv8_prefix_attn_fwd(s["q"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["table"], s["cu"],
                                       s["kv_lens"], s["cu_groups"], s["prefix_lens"], s["out"], s["params"], s["workspace"],
                                       lse=s["lse"])
    else:
        _plain_prefix(s)
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------------------ 64 bits
def _exact_qk_one(x, w, s):
    y = x.double()
    d, rot, a = y.shape[-1], s["rot"], s["start"]
    if w is not None:
        norm = torch.linalg.vector_norm(y, dim=-1, keepdim=True)
        y = y / torch.sqrt(norm * norm / d + s["eps"]) * w.double()
    z = y[..., a:a + rot]
    z = z.unflatten(-1, (rot // 2, 2)) if s["inter"] else torch.stack([z[..., :rot // 2], z[..., rot // 2:]], dim=-1)
    theta = torch.tensor([s["base"] ** (-2.0 * j / rot) for j in range(rot // 2)], dtype=torch.float64, device=x.device)
    turn = torch.polar(torch.ones_like(theta)[None, :].expand(x.shape[0], -1), s["pos"].double()[:, None] * theta[None, :])
    z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn[:, None, :])
    z = z.flatten(-2) if s["inter"] else torch.cat([z[..., 0], z[..., 1]], dim=-1)
    return torch.cat([y[..., :a], z, y[..., a + rot:]], dim=-1)


def _exact_gather(case, s):
    ctx, _ = _lens(case)
    codes = np.arange(256)
    e, m = (codes >> 3) & 15, codes & 7
    value = np.where(e > 0, (1 + m / 8.0) * 2.0 ** (e - 7.0), m * 2.0 ** -9) * np.where(codes > 127, -1.0, 1.0)
    pool, table = s["pool"].cpu().numpy(), s["table"].cpu().numpy()
    out = np.empty((sum(ctx), 576), np.float64)
    at = 0
    for r, n in enumerate(ctx):
        i = np.arange(n)
        rows = np.ascontiguousarray(pool[table[r, i // case["page"]].astype(np.int64) * case["page"] + i % case["page"]])
        scale = np.ascontiguousarray(rows[:, 512:528]).view(np.float32).astype(np.float64)
        out[at:at + n, :512] = value[rows[:, :512]] * np.repeat(scale, 128, axis=1)
        bits = np.ascontiguousarray(rows[:, 528:]).view(np.uint16).astype(np.uint32) << 16
        out[at:at + n, 512:] = bits.view(np.float32)
        at += n
    return {"out": torch.from_numpy(out)}


def _exact_mla(case, s):
    if work(case)["flops"] > 2e12:
        return None
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device="cuda")
    kv, q = _lens(case)
    cu, ck = _prefix(q), _prefix(kv)
    for r in range(case["n_req"]):
        a, b, c, e = cu[r], cu[r + 1], ck[r], ck[r + 1]
        hidden = torch.ones((q[r], kv[r]), dtype=torch.bool, device="cuda").triu(kv[r] - q[r] + 1)
        rope = s["k_rope"][c:e].double()
        for hh in range(case["h"]):
            key = torch.cat([s["k_nope"][c:e, hh].double(), rope], dim=1)
            z = torch.einsum("id,jd->ij", s["q"][a:b, hh].double(), key) / math.sqrt(192.0)
            z = torch.where(hidden, torch.full_like(z, -math.inf), z)
            out[a:b, hh] = torch.einsum("ij,jd->id", torch.softmax(z, dim=-1), s["v"][c:e, hh].double())
            lse[a:b, hh] = torch.logsumexp(z, dim=-1)
    return {"out": out, "lse": lse}


def _exact_prefix(case, s):
    if work(case)["flops"] > 2e12 or case["n_req"] * case["h"] > 2048:
        return None
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device="cuda")
    kv, q, _, _ = _lens(case)
    cu = _prefix(q)
    h, g, page = case["h"], case["h_q"] // case["h"], case["page"]
    for r in range(case["n_req"]):
        ids = s["table"][r, :_cdiv(kv[r], page)].long()
        a, b = cu[r], cu[r + 1]
        hidden = torch.arange(kv[r], device="cuda")[None, :] > torch.arange(kv[r] - q[r], kv[r], device="cuda")[:, None]
        k = s["k_pool"][ids].view(torch.float8_e4m3fn).double() * s["k_scale"][ids].double()[:, :, None, None]
        v = s["v_pool"][ids].view(torch.float8_e4m3fn).double() * s["v_scale"][ids].double()[:, :, None, None]
        k, v = (x.transpose(0, 1).reshape(h, -1, case["d"])[:, :kv[r]] for x in (k, v))
        qs = s["q"][a:b].double().unflatten(1, (h, g))
        z = torch.einsum("ihgd,hjd->hgij", qs, k) / math.sqrt(case["d"])
        z = torch.where(hidden[None, None], torch.full_like(z, -math.inf), z)
        out[a:b] = torch.einsum("hgij,hjd->ihgd", torch.softmax(z, dim=-1), v).flatten(1, 2)
        lse[a:b] = torch.logsumexp(z, dim=-1).permute(2, 0, 1).flatten(1, 2)
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "qk":
        both = {"q": _exact_qk_one(s["q"], s["q_w"], s)}
        if s["k"] is not None:
            both["k"] = _exact_qk_one(s["k"], s["k_w"], s)
        return both
    return {"gather": _exact_gather, "mla": _exact_mla, "prefix": _exact_prefix}[s["op"]](case, s)
