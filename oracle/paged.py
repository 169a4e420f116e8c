"""The paged 8-bit cache in float64 and plain loops (oracle; test infrastructure only):
the page map of a serving step, the insert, and the attention over the cache, restated
from their definitions (include/dsa_page_map.h, include/dsa_kv8.h).
"""

from __future__ import annotations

import math

import numpy as np

from . import codecs

OUT_OF_PAGES, TABLE_FULL, TOKENS_FULL = 8, 16, 32


def page_map(ctx, new, table, free, page, n_tokens):
    """(table, cu, kv_lens, positions, slots, token_req, info), one token at a time."""
    table = np.array(table, dtype=np.int32)
    cols = table.shape[1]
    cu, kv, status, taken = [0], [], 0, 0
    pos = np.zeros(n_tokens, np.int32)
    slots = np.full(n_tokens, -1, np.int64)
    req = np.full(n_tokens, -1, np.int32)
    t = 0
    for r, (c, w) in enumerate(zip(ctx, new)):
        c, w = max(int(c), 0), max(int(w), 0)
        if -(-(c + w) // page) > cols or c + w > 2 ** 31 - 1:
            status |= TABLE_FULL
        for i in range(min(-(-c // page), cols), min(-(-(c + w) // page), cols)):
            p = int(free[taken]) if taken < len(free) else -1
            if p < 0:
                status |= OUT_OF_PAGES
            table[r, i] = max(p, -1)
            taken += 1
        if w > 0 and c % page and c // page < cols and table[r, c // page] < 0:
            status |= OUT_OF_PAGES
        for i in range(min(w, n_tokens - t)):
            q = c + i
            pos[t], req[t] = min(q, 2 ** 31 - 1), r
            if q // page < cols and table[r, q // page] >= 0:
                slots[t] = int(table[r, q // page]) * page + q % page
            t += 1
        if cu[-1] + w > n_tokens:
            status |= TOKENS_FULL
        cu.append(min(cu[-1] + w, n_tokens))
        kv.append(min(c + w, 2 ** 31 - 1))
    return (table, np.array(cu, np.int32), np.array(kv, np.int32), pos, slots, req,
            np.array([min(taken, len(free)), status], np.int32))


def page_scale(amax: float) -> float:
    """Least power of two s with amax <= 448 s, within [2^-64, 2^64]."""
    e = -64
    while e < 64 and amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def kv8_insert(pool, scale, x, slots):
    """One pool: codes uint8 [n_pages, h, page, d], scales fp32 [n_pages, h], x float64
    [n, h, d]; returns new (pool, scale)."""
    pool, scale = pool.copy(), scale.copy()
    n_pages, h, page, _ = pool.shape
    i = 0
    while i < len(slots):
        if slots[i] < 0 or slots[i] >= n_pages * page:
            i += 1
            continue
        j = i + 1
        while j < len(slots) and slots[j] == slots[j - 1] + 1 and slots[j] % page != 0 and slots[j] < n_pages * page:
            j += 1
        pg, o0 = divmod(int(slots[i]), page)
        for hh in range(h):
            run = np.abs(x[i:j, hh])
            s = page_scale(float(np.max(run, initial=0.0, where=np.isfinite(run))))
            old = float(scale[pg, hh])
            if o0 > 0 and old >= s:
                s = old
            elif o0 > 0:
                v = codecs.e4m3_decode(pool[pg, hh, :o0])
                pool[pg, hh, :o0] = codecs.e4m3_encode(v * (old / s))
            scale[pg, hh] = s
            pool[pg, hh, o0:o0 + j - i] = codecs.e4m3_encode(x[i:j, hh] / s)
        i = j
    return pool, scale


def kv8_attention(q, k_pool, v_pool, k_scale, v_scale, table, cu, kv_lens, softmax_scale, window=0):
    """q float64 [n, h_q, d].  Returns (out, lse, error terms): out and lse NaN for rows of no request; the
    terms are what an error bound needs, see below."""
    n, h_q, d = q.shape
    n_pages, h, page, _ = k_pool.shape
    g = h_q // h
    out = np.full((n, h_q, d), np.nan)
    lse = np.full((n, h_q), np.nan)
    # sum_j p_j |v_j|;  max_j p_j v_scale_j * sum_j |code_j|;  max_j sum_i |q_i k_ij| * softmax_scale
    mass, tiny, size = np.zeros((n, h_q, d)), np.zeros((n, h_q, d)), np.zeros((n, h_q))
    for r in range(len(kv_lens)):
        a, b, kv = int(cu[r]), int(cu[r + 1]), min(int(kv_lens[r]), table.shape[1] * page)
        if b <= a:
            continue
        at = np.arange(kv)
        ids = table[r, at // page].astype(np.int64) if kv else np.zeros(0, np.int64)
        there = (ids >= 0) & (ids < n_pages)
        pos_all = np.arange(kv - (b - a), kv)
        seen_any = there & (at <= pos_all[-1])
        if window > 0:
            seen_any &= at > pos_all[0] - window
        js = at[seen_any]
        ids = ids[seen_any]
        for hh in range(h):
            kc = codecs.e4m3_decode(k_pool[ids, hh, js % page])
            vc = codecs.e4m3_decode(v_pool[ids, hh, js % page])
            ks, vs = k_scale[ids, hh].astype(np.float64)[:, None], v_scale[ids, hh].astype(np.float64)[:, None]
            for i in range(b - a):
                p = kv - (b - a) + i
                m = js <= p
                if window > 0:
                    m &= js > p - window
                for head in range(hh * g, hh * g + g):
                    if not m.any():
                        out[a + i, head], lse[a + i, head] = 0.0, -np.inf
                        continue
                    k = kc[m] * ks[m]
                    z = k @ q[a + i, head] * softmax_scale
                    top = z.max()
                    e = np.exp(z - top)
                    w = e / e.sum()
                    out[a + i, head] = w @ (vc[m] * vs[m])
                    lse[a + i, head] = top + math.log(e.sum())
                    mass[a + i, head] = w @ np.abs(vc[m] * vs[m])
                    tiny[a + i, head] = (w * vs[m][:, 0]).max() * np.abs(vc[m]).sum(axis=0)
                    size[a + i, head] = (np.abs(k) @ np.abs(q[a + i, head])).max() * abs(softmax_scale)
    return out, lse, (mass, tiny, size)
