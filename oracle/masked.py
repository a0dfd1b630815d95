"""fp64 oracle of masked paged attention and of the head norm, rotation and cache write (CPU,
numpy; test infrastructure only).  Written from the definitions in include/inkling_attn.h."""
from __future__ import annotations

import math

import numpy as np


def _bf(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def visible(p, L, begin, end, window):
    """[first, last + 1) of the keys the token at position p sees."""
    lo = max(0, 0 if begin is None else int(begin), p - window + 1 if window > 0 else 0)
    hi = min(L, p + 1 if end is None else int(end))
    return lo, max(lo, hi)


def attention(*, num_q_heads, num_kv_heads, head_dim, page_size, window, sm_scale, cu_q, seq_lens, q_bits, k_bits,
              v_bits, block_table, softcap=0.0, key_begin=None, key_end=None, slopes=None):
    """(out [T, Hq, D], lse [T, Hq], mag [T, Hq, D], smag [T, Hq]).  For error bounds: mag is
    sum_k softmax(s)_k |V[k]|, smag the largest sum of magnitudes that went into a score.  Rows of no
    sequence are NaN."""
    T, Hq, D, G = q_bits.shape[0], num_q_heads, head_dim, num_q_heads // num_kv_heads
    out = np.full((T, Hq, D), np.nan)
    mag = np.full((T, Hq, D), np.nan)
    lse = np.full((T, Hq), np.nan)
    smag = np.zeros((T, Hq))
    q = _bf(q_bits)
    num_pages = k_bits.shape[0]
    for b in range(len(seq_lens)):
        t0, t1, L = int(cu_q[b]), int(cu_q[b + 1]), int(seq_lens[b])
        for t in range(t0, t1):
            p = L - (t1 - t0) + (t - t0)
            lo, hi = visible(p, L, None if key_begin is None else key_begin[t], None if key_end is None else key_end[t],
                             window)
            if t1 - t0 > L:
                hi = lo
            keys = np.arange(lo, hi)
            keys = keys[keys // page_size < block_table.shape[1]]
            page = block_table[b, keys // page_size]
            ok = (page >= 0) & (page < num_pages)
            keys, page = keys[ok], page[ok]
            for h in range(Hq):
                out[t, h] = mag[t, h] = 0.0
                lse[t, h] = -np.inf
                if keys.size == 0:
                    continue
                g = h // G
                K, V = _bf(k_bits[page, g, keys % page_size]), _bf(v_bits[page, g, keys % page_size])
                s = sm_scale * (K @ q[t, h])
                size = sm_scale * (np.abs(K) @ np.abs(q[t, h])) + softcap
                if softcap > 0:
                    s = softcap * np.tanh(s / softcap)
                if slopes is not None:
                    s = s - float(slopes[h]) * np.abs(p - keys)
                    size = size + abs(float(slopes[h])) * np.abs(p - keys)
                smag[t, h] = size.max()
                m = s.max()
                w = np.exp(s - m)
                tot = w.sum()
                lse[t, h] = m + math.log(tot)
                w = w / tot
                out[t, h] = w @ V
                mag[t, h] = w @ np.abs(V)
    return out, lse, mag, smag


def norm_rope(x, pos, w, eps, inv_freq, layout, rot_scale):
    """x [n, H, D] fp64 at positions pos [n]: (result, magnitude of the terms that were added)."""
    y = x.copy()
    if w is not None:
        y = y / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    mag = np.abs(y)
    rot = 0 if inv_freq is None else 2 * len(inv_freq)
    if rot:
        ang = pos[:, None].astype(np.float64) * inv_freq.astype(np.float64)[None]
        c, s = rot_scale * np.cos(ang)[:, None], rot_scale * np.sin(ang)[:, None]
        i = np.arange(rot // 2)
        ia, ib = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
        a, b = y[..., ia], y[..., ib]
        z = y.copy()
        z[..., ia], z[..., ib] = a * c - b * s, b * c + a * s
        mag[..., ia] = mag[..., ib] = rot_scale * (np.abs(a) + np.abs(b))
        y = z
    return y, mag
