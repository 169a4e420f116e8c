"""Cases of the paged-cache operators: the page map (dsa_page_map), the insert into a cache held in 8 bits with one
scale per page and KV head (dsa_kv8_insert), and the attention that reads that cache (dsa_kv8_attn_fwd).

`run` computes them in elementary torch operations, or, where `own` is true, with the library's entry points; `exact`
restates each definition in 64 bits.

Definitions.  P = page size, h = h_kv, g = h_q / h_kv.
  map     cu = prefix sum of new; request r's tokens sit at positions ctx[r] + i; pages old[r] = ceil(ctx[r] / P) are in
          its table row, the others up to ceil((ctx[r] + new[r]) / P) are taken from the free list in request order;
          slot = page * P + position % P.  Rows behind the last request: position 0, slot -1, request -1.
  insert  pool row of a slot: page slot / P, offset slot % P.  The tokens of one page are a run of consecutive slots
          from offset o0.  Per page and head: s = the least power of two >= 2^-64 with max|x| <= 448 s over the run, and
          with o0 > 0 at least the page's old scale; the rows before o0 are rescaled by old / s where s grew; codes are
          E4M3 values nearest to x / s (ties to even).
  attn    query i of request r is at position kv_len[r] - q_len[r] + i and sees the keys at positions j <= its own (and,
          with a window W > 0, j > its own - W); out = softmax(scale * q.k) v, lse = the natural-log sum-exp."""

import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # the smallest decode step: a few requests, one new token each, latency alone
        {"name": "map_decode_16", "op": "map", "n_req": 16, "ctx_max": 4096, "new_max": 1, "page": 64, "pad": 0, "lens": 1},
        # a large decode step replayed at a fixed padded batch size, an odd request count
        {"name": "map_decode_1021_pad", "op": "map", "n_req": 1021, "ctx_max": 32768, "new_max": 1, "page": 16, "pad": 3, "lens": 2},
        # a prefill wave: few requests with many new tokens and many new pages
        {"name": "map_prefill_33", "op": "map", "n_req": 33, "ctx_max": 2048, "new_max": 4096, "page": 64, "pad": 0, "lens": 3},
        # decode: one new token per request, each into its own page
        {"name": "insert_decode_64", "op": "insert", "n_req": 64, "ctx_max": 32768, "new_max": 1, "h": 8, "d": 128, "page": 64, "dtype": "bf16", "lens": 4},
        # one prefill chunk of an odd length, fp16 keys and values
        {"name": "insert_prefill_2123", "op": "insert", "n_req": 1, "ctx_max": 1, "new_max": 2123, "h": 8, "d": 128, "page": 64, "dtype": "fp16", "lens": 5},
        # a prefill wave of ragged requests that continue half-filled pages
        {"name": "insert_prefill_65536", "op": "insert", "n_req": 32, "ctx_max": 1024, "new_max": 3967, "h": 8, "d": 128, "page": 32, "dtype": "bf16", "lens": 6},
        # one user's token against a long context: split over the whole GPU
        {"name": "attn_decode_1", "op": "attn", "n_req": 1, "q_max": 1, "kv_max": 32768, "h_q": 64, "h": 8, "d": 128, "page": 64, "window": 0, "dtype": "bf16", "lens": 7},
        # batched decode with ragged contexts: the cache's bytes bound it
        {"name": "attn_decode_64", "op": "attn", "n_req": 64, "q_max": 1, "kv_max": 32768, "h_q": 64, "h": 8, "d": 128, "page": 64, "window": 0, "dtype": "bf16", "lens": 8},
        # many short conversations of a small model under a sliding window, fp16, small pages
        {"name": "attn_decode_1024", "op": "attn", "n_req": 1024, "q_max": 1, "kv_max": 2123, "h_q": 16, "h": 2, "d": 64, "page": 16, "window": 640, "dtype": "fp16", "lens": 9},
        # drafted tokens verified at once: four or fewer queries per request
        {"name": "attn_verify_48", "op": "attn", "n_req": 48, "q_max": 4, "kv_max": 8192, "h_q": 32, "h": 8, "d": 128, "page": 32, "window": 0, "dtype": "bf16", "lens": 10},
        # one prefill chunk of an odd length from the start of a sequence
        {"name": "attn_prefill_2123", "op": "attn", "n_req": 1, "q_max": 2123, "kv_max": 2123, "h_q": 64, "h": 8, "d": 128, "page": 64, "window": 0, "dtype": "bf16", "lens": 11},
        # ragged chunks of several requests behind contexts of their own
        {"name": "attn_chunks_6", "op": "attn", "n_req": 6, "q_max": 2048, "kv_max": 8192, "h_q": 32, "h": 4, "d": 128, "page": 64, "window": 0, "dtype": "bf16", "lens": 12},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["map", "insert", "attn", "attn"])
    page = rng.choice([16, 32, 64, 128])
    lens = rng.randrange(1, 1 << 20)
    if op == "map":
        n_req = _log_int(rng, 1, 2048)
        new_max = rng.choice([1, 1, _log_int(rng, 2, max(2, min(8192, 131072 // n_req)))])
        return {"op": op, "n_req": n_req, "ctx_max": _log_int(rng, 1, 32768), "new_max": new_max, "page": page,
                "pad": rng.choice([0, 0, rng.randrange(1, 100)]), "lens": lens}
    dtype = rng.choice(["bf16", "fp16"])
    d = rng.choice([64, 128])
    h = rng.choice([1, 2, 3, 4, 8])
    if op == "insert":
        n_req = _log_int(rng, 1, 512)
        new_max = rng.choice([1, _log_int(rng, 2, max(2, min(8192, 98304 // n_req)))])
        return {"op": op, "n_req": n_req, "ctx_max": _log_int(rng, 1, 8192), "new_max": new_max, "h": h, "d": d,
                "page": page, "dtype": dtype, "lens": lens}
    g = rng.choice([1, 2, 4, 5, 8, 12, 16])
    window = rng.choice([0, 0, _log_int(rng, 1, 4096)])
    if rng.random() < 0.5:   # decode and verification
        n_req = _log_int(rng, 1, 512)
        kv_max = _log_int(rng, 16, max(16, min(32768, 1 << 20 >> max(0, n_req.bit_length() - 1))))
        q_max = min(kv_max, rng.choice([1, 1, 2, 4, 7]))
    else:                    # prefill
        n_req = rng.choice([1, 2, 3, 5])
        kv_max = _log_int(rng, 64, 4096)
        q_max = _log_int(rng, 8, kv_max)
        g = min(g, 8)
    return {"op": op, "n_req": n_req, "q_max": q_max, "kv_max": kv_max, "h_q": h * g, "h": h, "d": d, "page": page,
            "window": window, "dtype": dtype, "lens": lens}


# ------------------------------------------------------------------------------ sizes
def _lens(case):
    """Request lengths of a case: (before, new) per request.  They belong to the case, not to the seed."""
    r = random.Random(case["lens"])
    n = case["n_req"]
    if case["op"] == "attn":
        q = [r.randint(max(1, case["q_max"] // 2), case["q_max"]) for _ in range(n)]
        kv = [r.randint(a, case["kv_max"]) for a in q]
        q[0], kv[0] = case["q_max"], case["kv_max"]
        return [b - a for a, b in zip(q, kv)], q
    new = [case["new_max"]] * n if case["new_max"] == 1 else [r.randint(0, case["new_max"]) for _ in range(n)]
    new[0] = case["new_max"]
    return [r.randint(0, case["ctx_max"]) for _ in range(n)], new


def _cdiv(a, b):
    return -(-a // b)


def _prefix(v):
    return [0] + list(np.cumsum(np.asarray(v, dtype=np.int64)).tolist())


def _pairs(kv, q, window):
    """Visible (query, key) pairs of one request."""
    pos = np.arange(kv - q, kv, dtype=np.int64) + 1
    return int(np.minimum(pos, window if window > 0 else kv).sum())


def work(case):
    ctx, new = _lens(case)
    n, t, page = case["n_req"], sum(new), case["page"]
    pages = sum(_cdiv(a + b, page) - _cdiv(a, page) for a, b in zip(ctx, new))
    if case["op"] == "map":
        # lengths in; cu, kv_lens out; one page id in and one table entry out per new page; 16 bytes per token
        return {"bytes": 16 * n + 8 * pages + 16 * (t + case["pad"]), "flops": 0}
    if case["op"] == "insert":
        runs = sum(_cdiv(a + b, page) - a // page for a, b in zip(ctx, new) if b)
        return {"bytes": t * case["h"] * case["d"] * 2 * 3 + 8 * t + runs * case["h"] * 16, "flops": 4 * t * case["h"] * case["d"]}
    pairs = sum(_pairs(a + b, b, case["window"]) for a, b in zip(ctx, new))
    w = case["window"]
    live = sum(min(a + b, w + b - 1) if w > 0 else a + b for a, b in zip(ctx, new))
    return {"bytes": live * case["h"] * case["d"] * 2 + t * case["h_q"] * (4 * case["d"] + 4) + _cdiv(live, page) * (4 + 8 * case["h"]),
            "flops": 4 * pairs * case["h_q"] * case["d"]}


# ------------------------------------------------------------------------------ inputs
def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _tables(case, ctx, total, gen):
    """A random page order and, for each request, its row of pages (-1 behind them): (table, the pages not used, page count)."""
    page = case["page"]
    used = [_cdiv(a, page) for a in total]
    cols = max(1, max(_cdiv(a + b, page) for a, b in zip(ctx, case["_new"])))
    spare = sum(_cdiv(a + b, page) for a, b in zip(ctx, case["_new"])) - sum(used) + 5
    n_pages = sum(used) + spare
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    start = _ints(_prefix(used)[:-1], torch.int64)
    col = torch.arange(cols, device="cuda")
    at = (start[:, None] + col[None, :]).clamp_(max=n_pages - 1)
    table = torch.where(col[None, :] < _ints(used)[:, None], order[at], torch.full_like(order[at], -1))
    return table.contiguous(), order[sum(used):].contiguous(), n_pages


def _cache(n_pages, h, page, d, gen):
    """A pool as the insert leaves it: keys or values of a magnitude of their own for each page and head, with the
    power-of-two scale of that page."""
    pool = torch.empty((n_pages, h, page, d), dtype=torch.uint8, device="cuda")
    mag = torch.exp2(torch.randint(-2, 2, (n_pages, h, 1, 1), generator=gen, device="cuda").float())
    step = max(1, (1 << 26) // (h * page * d))
    for a in range(0, n_pages, step):
        x = torch.randn((min(step, n_pages - a), h, page, d), generator=gen, device="cuda")
        pool[a:a + step] = (x * 64.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return pool, (mag / 64.0).reshape(n_pages, h).contiguous()


def prepare(case, seed):
    case = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) & 0x7FFFFFFF)
    ctx, new = _lens(case)
    case["_new"] = new
    n, t, page = case["n_req"], sum(new), case["page"]
    total = [a + b for a, b in zip(ctx, new)]
    st = {"op": case["op"], "page": page}
    if case["op"] == "map":
        table, free, _ = _tables(case, ctx, ctx, gen)
        m = t + case["pad"]
        st |= {"ctx": _ints(ctx), "new": _ints(new), "table": table, "free": free, "n_tokens": m,
               "cu": torch.empty(n + 1, dtype=torch.int32, device="cuda"),
               "kv_lens": torch.empty(n, dtype=torch.int32, device="cuda"),
               "positions": torch.empty(m, dtype=torch.int32, device="cuda"),
               "slots": torch.empty(m, dtype=torch.int64, device="cuda"),
               "token_req": torch.empty(m, dtype=torch.int32, device="cuda"),
               "info": torch.empty(2, dtype=torch.int32, device="cuda")}
        return st
    table, _, n_pages = _tables(case, ctx, total, gen)
    h, d, dtype = case["h"], case["d"], DTYPES[case["dtype"]]
    st["k_pool"], st["k_scale"] = _cache(n_pages, h, page, d, gen)
    st["v_pool"], st["v_scale"] = _cache(n_pages, h, page, d, gen)
    if case["op"] == "insert":
        req = torch.repeat_interleave(torch.arange(n, device="cuda"), _ints(new, torch.int64))
        pos = torch.arange(t, device="cuda") - _ints(_prefix(new)[:-1], torch.int64)[req] + _ints(ctx, torch.int64)[req]
        st["slots"] = table[req, pos // page].to(torch.int64) * page + pos % page
        # the new rows of a packed qkv projection's output: a row pitch larger than the row
        kv = torch.randn((t, 2 * h + 1, d), generator=gen, device="cuda")
        kv[:, :, ::17] *= 6.0   # a few channels carry most of the magnitude
        kv = kv.to(dtype)
        st["k"], st["v"] = kv[:, :h], kv[:, h:2 * h]
        return st
    st |= {"q": (torch.randn((t, case["h_q"], d), generator=gen, device="cuda") * 2.0).to(dtype), "table": table,
           "cu": _ints(_prefix(new)), "kv_lens": _ints(total), "q_max": max(new), "window": case["window"],
           "scale": 1.0 / math.sqrt(d),
           "out": torch.empty((t, case["h_q"], d), dtype=dtype, device="cuda"),
           "lse": torch.empty((t, case["h_q"]), dtype=torch.float32, device="cuda")}
    if own:
        from top_sparse_mla_gb300 import native
        st["params"] = native.dsa_kv8_params_init(st["q"], st["k_pool"], table, max_q_len=st["q_max"], window=st["window"])
        st["workspace"] = torch.empty(native.dsa_kv8_attn_workspace_size(st["params"]), dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------------------ plain forms
def _plain_map(s):
    ctx, new, page, m = s["ctx"].long(), s["new"].long(), s["page"], s["n_tokens"]
    n, cols = s["table"].shape
    kv = ctx + new
    end = torch.cumsum(new, 0)
    cu = torch.cat([torch.zeros_like(end[:1]), end])
    old = (ctx + page - 1) // page
    take = (kv + page - 1) // page - old
    off = torch.cumsum(take, 0) - take
    col = torch.arange(cols, device="cuda")[None, :]
    i = col - old[:, None]
    fresh = (i >= 0) & (i < take[:, None])
    at = (off[:, None] + i).clamp(0, s["free"].numel() - 1)
    s["table"].copy_(torch.where(fresh, s["free"][at], s["table"]))
    t = torch.arange(m, device="cuda")
    req = torch.searchsorted(end, t, right=True)
    live = req < n
    r = req.clamp(max=n - 1)
    pos = torch.where(live, t - cu[r] + ctx[r], torch.zeros_like(t))
    slot = s["table"][r, (pos // page).clamp(max=cols - 1)].long() * page + pos % page
    s["cu"].copy_(cu)
    s["kv_lens"].copy_(kv)
    s["positions"].copy_(pos)
    s["slots"].copy_(torch.where(live, slot, torch.full_like(slot, -1)))
    s["token_req"].copy_(torch.where(live, req, torch.full_like(req, -1)))
    s["info"].copy_(torch.stack([take.sum(), torch.zeros_like(take.sum())]))


def _plain_insert_one(x, slots, pool, scale, page):
    p, o = slots // page, slots % page
    first = torch.ones_like(p, dtype=torch.bool)
    first[1:] = p[1:] != p[:-1]
    run = torch.cumsum(first.long(), 0) - 1
    pages, o0 = p[first], o[first]
    amax = torch.zeros((pages.numel(), x.shape[1]), dtype=torch.float32, device=x.device)
    amax.scatter_reduce_(0, run[:, None].expand(-1, x.shape[1]), x.float().abs().amax(dim=2), "amax")
    m, e = torch.frexp(amax)
    e = torch.where(m > 0.875, e - 8, e - 9)
    s = torch.exp2(torch.where(amax > 0, e.clamp(min=-64), torch.full_like(e, -64)).float())
    old = torch.where((o0 > 0)[:, None], scale[pages], torch.zeros_like(s))
    s = torch.maximum(s, old)
    rows = pool[pages].view(torch.float8_e4m3fn).float()
    moved = (rows * (old / s)[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    before = torch.arange(page, device=x.device)[None, None, :, None] < o0[:, None, None, None]
    pool[pages] = torch.where(before, moved, pool[pages])
    scale[pages] = s
    pool[p, :, o] = (x.float() / s[run][:, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_attn(s):
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
    j = torch.arange(k.shape[2], device="cuda")
    seen = j[None, None, :] <= pos[:, :, None]
    if s["window"] > 0:
        seen &= j[None, None, :] > pos[:, :, None] - s["window"]
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
    if s["op"] == "map":
        if own:
            native.dsa_page_map(s["ctx"], s["new"], s["table"], s["free"], s["page"], s["cu"], s["kv_lens"],
                                s["positions"], s["slots"], s["token_req"], s["info"])
        else:
            _plain_map(s)
        return {k: s[k] for k in ("table", "cu", "kv_lens", "positions", "slots", "token_req", "info")}
    if s["op"] == "insert":
        if own:
            native.dsa_kv8_insert(s["k"], s["v"], s["slots"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"])
        else:
            _plain_insert_one(s["k"], s["slots"], s["k_pool"], s["k_scale"], s["page"])
            _plain_insert_one(s["v"], s["slots"], s["v_pool"], s["v_scale"], s["page"])
        return {"k_pool": s["k_pool"].view(torch.float8_e4m3fn), "v_pool": s["v_pool"].view(torch.float8_e4m3fn),
                "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if own:
        native.dsa_kv8_attn_fwd(s["q"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["table"], s["cu"],
                                s["kv_lens"], s["out"], s["params"], s["workspace"], lse=s["lse"])
    else:
        _plain_attn(s)
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------------------ 64 bits
def _nearest_e4m3(x):
    """The E4M3 value nearest to each float64 value, ties to the even code, saturating at 448."""
    a = np.minimum(np.abs(x), 448.0)
    step = np.exp2(np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -6.0) - 3.0)
    return np.copysign(np.minimum(np.rint(a / step) * step, 448.0), x)


def _exact_insert_one(x, slots, pool, scale, page):
    pool = pool.view(torch.float8_e4m3fn).float().cpu().numpy().astype(np.float64)
    scale = scale.double().cpu().numpy()
    x = x.double().cpu().numpy()
    slots = slots.cpu().numpy()
    p = slots // page
    cuts = np.concatenate([[0], np.nonzero(np.diff(p))[0] + 1, [len(p)]])
    for a, b in zip(cuts[:-1], cuts[1:]):
        pg, o = int(p[a]), int(slots[a] % page)
        for hh in range(x.shape[1]):
            amax = np.abs(x[a:b, hh]).max()
            e = -64
            if amax > 0:
                e = max(e, int(math.ceil(math.log2(amax / 448.0) - 1e-12)))
                while e > -64 and amax <= 448.0 * 2.0 ** (e - 1):
                    e -= 1
                while amax > 448.0 * 2.0 ** e:
                    e += 1
            s = 2.0 ** e
            if o > 0 and scale[pg, hh] >= s:
                s = scale[pg, hh]
            elif o > 0:
                pool[pg, hh, :o] = _nearest_e4m3(pool[pg, hh, :o] * (scale[pg, hh] / s))
            scale[pg, hh] = s
            pool[pg, hh, o:o + b - a] = _nearest_e4m3(x[a:b, hh] / s)
    return torch.from_numpy(pool), torch.from_numpy(scale)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "map":
        ctx, new, page = s["ctx"].tolist(), s["new"].tolist(), s["page"]
        table, free = s["table"].cpu().numpy().copy(), s["free"].tolist()
        cu, kv, pos, slots, reqs, taken = [0], [], [], [], [], 0
        for r, (c, w) in enumerate(zip(ctx, new)):
            for i in range(_cdiv(c, page), _cdiv(c + w, page)):
                table[r, i] = free[taken]
                taken += 1
            p = np.arange(c, c + w)
            pos += p.tolist()
            slots += (table[r, p // page].astype(np.int64) * page + p % page).tolist()
            reqs += [r] * w
            cu.append(cu[-1] + w)
            kv.append(c + w)
        pad = s["n_tokens"] - len(pos)
        as_int = lambda v, t: torch.tensor(v, dtype=t)  # noqa: E731
        return {"table": torch.from_numpy(table), "cu": as_int(cu, torch.int32), "kv_lens": as_int(kv, torch.int32),
                "positions": as_int(pos + [0] * pad, torch.int32), "slots": as_int(slots + [-1] * pad, torch.int64),
                "token_req": as_int(reqs + [-1] * pad, torch.int32), "info": as_int([taken, 0], torch.int32)}
    if s["op"] == "insert":
        if case["h"] * case["d"] * s["slots"].numel() > 1 << 26:
            return None   # minutes on the host
        kp, ks = _exact_insert_one(s["k"], s["slots"], s["k_pool"], s["k_scale"], s["page"])
        vp, vs = _exact_insert_one(s["v"], s["slots"], s["v_pool"], s["v_scale"], s["page"])
        return {"k_pool": kp, "v_pool": vp, "k_scale": ks, "v_scale": vs}
    _, new = _lens(case)
    cu, kv = s["cu"].tolist(), s["kv_lens"].tolist()
    if sum(_pairs(b, a, 0) for a, b in zip(new, kv)) * case["h_q"] * case["d"] > 1 << 40 or case["n_req"] > 1024:
        return None
    h, g, page = case["h"], case["h_q"] // case["h"], s["page"]
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device="cuda")
    for r in range(case["n_req"]):
        ids = s["table"][r, :_cdiv(kv[r], page)].long()
        a, b = cu[r], cu[r + 1]
        pos = torch.arange(kv[r] - (b - a), kv[r], device="cuda")[:, None]
        j = torch.arange(kv[r], device="cuda")[None, :]
        hidden = j > pos
        if case["window"] > 0:
            hidden = hidden | (pos - j >= case["window"])
        for hh in range(h):
            k = (s["k_pool"][ids, hh].view(torch.float8_e4m3fn).double() * s["k_scale"][ids, hh].double()[:, None, None]).flatten(0, 1)[:kv[r]]
            v = (s["v_pool"][ids, hh].view(torch.float8_e4m3fn).double() * s["v_scale"][ids, hh].double()[:, None, None]).flatten(0, 1)[:kv[r]]
            z = torch.einsum("igd,jd->gij", s["q"][a:b, hh * g:(hh + 1) * g].double(), k) / math.sqrt(case["d"])
            z = torch.where(hidden[None], torch.full_like(z, -math.inf), z)
            out[a:b, hh * g:(hh + 1) * g] = torch.einsum("gij,jd->igd", torch.softmax(z, dim=-1), v)
            lse[a:b, hh * g:(hh + 1) * g] = torch.logsumexp(z, dim=-1).T
    return {"out": out, "lse": lse}
