"""fp64 oracle of the operators on trees of drafted tokens (CPU, numpy; test infrastructure only).  Written
from the definitions in include/inkling_attn.h."""
from __future__ import annotations

import numpy as np


def _bf(bits):
    return (np.asarray(bits).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def ways(parents):
    """For each token of one sequence the tokens from the root to it."""
    got = []
    for i, p in enumerate(parents):
        got.append((list(got[p]) if 0 <= p < i else []) + [i])
    return got


def plan(parents, history, words):
    """(positions, ancestor bits [n, words]) of one sequence."""
    bits = np.zeros((len(parents), words), np.uint32)
    way = ways(parents)
    for i, w in enumerate(way):
        for j in w:
            bits[i, j // 32] |= np.uint32(1) << np.uint32(j % 32)
    return np.array([history + len(w) - 1 for w in way], np.int64), bits


def attention(*, num_q_heads, num_kv_heads, head_dim, page_size, window, sm_scale, cu_q, seq_lens, q_bits, k_bits,
              v_bits, block_table, positions, ancestors, rel=None, softcap=0.0, slopes=None):
    """(out [T, Hq, D], lse [T, Hq], mag [T, Hq, D], smag [T, Hq]): as oracle.masked.attention, for rows that see the
    history and the drafted tokens whose bits are set.  ancestors is uint32 [T, words], rel fp64 [T, Hq, E]."""
    T, Hq, D, G = q_bits.shape[0], num_q_heads, head_dim, num_q_heads // num_kv_heads
    out, mag = np.full((T, Hq, D), np.nan), np.full((T, Hq, D), np.nan)
    lse, smag = np.full((T, Hq), np.nan), np.zeros((T, Hq))
    q = _bf(q_bits)
    words = ancestors.shape[1]
    for b in range(len(seq_lens)):
        t0, t1, L = int(cu_q[b]), int(cu_q[b + 1]), int(seq_lens[b])
        n, H = t1 - t0, L - (t1 - t0)
        out[t0:t1] = mag[t0:t1] = 0.0
        lse[t0:t1] = -np.inf
        if n == 0 or n > L or n > 32 * words:
            continue
        p = np.maximum(positions[t0:t1].astype(np.int64), H)
        keys = np.arange(L)
        pos = np.concatenate((np.arange(H), p))
        see = np.ones((n, L), bool)
        for j in range(n):
            see[:, H + j] = (ancestors[t0:t1, j // 32] >> np.uint32(j % 32)) & 1
        if window > 0:
            see &= p[:, None] - pos[None] <= window - 1
        col = keys // page_size
        page = np.where(col < block_table.shape[1], block_table[b, np.minimum(col, block_table.shape[1] - 1)], -1)
        see &= ((page >= 0) & (page < k_bits.shape[0]))[None]
        used = see.any(0)
        keys, page, pos, see = keys[used], page[used], pos[used], see[:, used]
        if keys.size == 0:
            continue
        far = np.abs(p[:, None] - pos[None])
        for g in range(num_kv_heads):
            K, V = _bf(k_bits[page, g, keys % page_size]), _bf(v_bits[page, g, keys % page_size])
            for h in range(g * G, (g + 1) * G):
                s = sm_scale * (q[t0:t1, h] @ K.T)
                size = abs(sm_scale) * (np.abs(q[t0:t1, h]) @ np.abs(K).T) + softcap
                if softcap > 0:
                    s = softcap * np.tanh(s / softcap)
                if slopes is not None:
                    s = s - float(slopes[h]) * far
                    size = size + abs(float(slopes[h])) * far
                if rel is not None:
                    r = np.take_along_axis(rel[t0:t1, h], np.minimum(far, rel.shape[-1] - 1), 1)
                    s, size = s + r, size + np.abs(r)
                for i in range(n):
                    on = see[i]
                    if not on.any():
                        continue
                    si = s[i, on]
                    m = si.max()
                    w = np.exp(si - m)
                    lse[t0 + i, h] = m + np.log(w.sum())
                    w /= w.sum()
                    smag[t0 + i, h] = size[i, on].max()
                    out[t0 + i, h] = w @ V[on]
                    mag[t0 + i, h] = w @ np.abs(V[on])
    return out, lse, mag, smag


def conv(x_bits, state_bits, parents, w):
    """The convolution of one sequence's rows x [n, Hkv, D] along the ways to the root: (y, sum of |terms|), with the
    state's rows [ks - 1, Hkv, D] before every root."""
    ks = w.shape[-1]
    x, w = _bf(x_bits), np.asarray(w, np.float64)
    rows = np.concatenate((_bf(state_bits), x)) if ks > 1 else x
    y, mag = np.zeros_like(x), np.zeros_like(x)
    for i, way in enumerate(ways(parents)):
        line = list(range(ks - 1)) + [ks - 1 + j for j in way]
        for j, r in enumerate(line[-ks:]):
            y[i] += w[..., j] * rows[r]
            mag[i] += np.abs(w[..., j] * rows[r])
    return y, mag


def conv_state(x_bits, state_bits, path):
    """The state (bits) of one sequence behind the accepted path."""
    keep = state_bits.shape[0]
    return np.concatenate((state_bits, x_bits[np.asarray(path, np.int64)]))[len(path):][:keep]


def accepted(path, m, n):
    """The path of m entries if it is one of n drafted tokens, else an empty one."""
    if m < 0 or m > len(path):
        return []
    p = [int(x) for x in path[:m]]
    ok = all(0 <= x < n for x in p) and all(a < b for a, b in zip(p, p[1:]))
    return p if ok else []


def commit(cache, block_table, page_size, num_pages, history, path):
    """The rows of one sequence's path moved behind its history, in place (cache [num_pages, Hkv, P, D], any type)."""
    def at(key):
        c = key // page_size
        page = int(block_table[c]) if c < len(block_table) else -1
        return (page, key % page_size) if 0 <= page < num_pages else None
    for j, i in enumerate(path):
        src, dst = at(history + i), at(history + j)
        if i != j and src and dst:
            cache[dst[0], :, dst[1]] = cache[src[0], :, src[1]]
