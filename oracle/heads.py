"""What stands in front of a layer's attention, and the expanded latent attention, in float64 and plain loops (oracle; test
infrastructure only): the norm and rotation of heads (include/dsa_qk_norm_rope.h), latent rows read back from the cache
(include/dsa_kv_gather.h), attention with expanded latent keys and values (include/dsa_mla_prefill.h).
"""

from __future__ import annotations

import math

import numpy as np

from . import codecs


def norm_rope(x, w, positions, rotary_dim, rotary_start=0, interleaved=False, eps=1e-6, base=10000.0):
    """x float64 [n, h, d]; w float64 [d] or None.  Returns the result and, for each value, |a| + |b| of its rotary
    pair (|y| outside them): what an error of the rotation is relative to."""
    y = np.array(x, dtype=np.float64)
    if w is not None:
        y = y / np.sqrt((y * y).mean(axis=-1, keepdims=True) + eps) * w
    out, size = y.copy(), np.abs(y)
    for t, p in enumerate(positions):
        for i in range(rotary_dim // 2):
            # the angle's turns, in exact arithmetic up to the frequency's own rounding
            angle = math.fmod(int(p) * (base ** (-2.0 * i / rotary_dim)), 2.0 * math.pi)
            c, s = math.cos(angle), math.sin(angle)
            at = (rotary_start + 2 * i, rotary_start + 2 * i + 1) if interleaved else (rotary_start + i, rotary_start + i + rotary_dim // 2)
            a, b = y[t, :, at[0]], y[t, :, at[1]]
            out[t, :, at[0]], out[t, :, at[1]] = a * c - b * s, a * s + b * c
            size[t, :, at[0]] = size[t, :, at[1]] = np.abs(a) + np.abs(b)
    return out, size


def kv_gather(pool, table, cu, lens, page, n_out):
    """(rows float64 [n_out, 576], NaN where nothing is written; whether a row had no place in the pool)."""
    out, missing = np.full((n_out, 576), np.nan), False
    for r in range(len(cu) - 1):
        a, b = (min(max(int(c), 0), n_out) for c in cu[r:r + 2])
        for i in range(min(b - a, max(int(lens[r]), 0)) if lens is not None else b - a):
            p = int(table[r, i // page]) if i // page < table.shape[1] else -1
            row = p * page + i % page
            if p < 0 or row >= len(pool):
                out[a + i], missing = 0.0, True
                continue
            scale = pool[row, 512:528].copy().view("<f4").astype(np.float64)
            out[a + i, :512] = codecs.e4m3_decode(pool[row, :512]) * np.repeat(scale, 128)
            out[a + i, 512:] = (pool[row, 528:].copy().view("<u2").astype(np.uint32) << 16).view(np.float32)
    return out, missing


def latent_attention(q, k_nope, k_rope, v, cu_q, cu_kv, softmax_scale):
    """q float64 [n, h, 192], k_nope and v [m, h, 128], k_rope [m, 64].  Returns (out, lse, (mass, size)): out and lse NaN for
    rows of no request; mass = sum_j p_j |v_j|, size = max_j sum_i |q_i k_ij| * softmax_scale."""
    n, h, _ = q.shape
    out, lse = np.full((n, h, 128), np.nan), np.full((n, h), np.nan)
    mass, size = np.zeros((n, h, 128)), np.zeros((n, h))
    for r in range(len(cu_q) - 1):
        a, b = (min(max(int(c), 0), n) for c in cu_q[r:r + 2])
        c, e = (min(max(int(x), 0), len(k_rope)) for x in cu_kv[r:r + 2])
        for i in range(b - a):
            m = min((e - c) - (b - a) + i + 1, e - c)
            for hh in range(h):
                if m <= 0:
                    out[a + i, hh], lse[a + i, hh] = 0.0, -np.inf
                    continue
                k = np.concatenate([k_nope[c:c + m, hh], k_rope[c:c + m]], axis=1)
                z = k @ q[a + i, hh] * softmax_scale
                top = z.max()
                w = np.exp(z - top)
                total = w.sum()
                w = w / total
                out[a + i, hh], lse[a + i, hh] = w @ v[c:c + m, hh], top + math.log(total)
                mass[a + i, hh] = w @ np.abs(v[c:c + m, hh])
                size[a + i, hh] = (np.abs(k) @ np.abs(q[a + i, hh])).max() * abs(softmax_scale)
    return out, lse, (mass, size)
