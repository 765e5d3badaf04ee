"""Attention of drafted tokens and the move of accepted ones in float64 (the
definitions of q4g128_attn_tree and q4g128_cache_keep in include/q4g128.h), one
token and one head at a time.
"""
from __future__ import annotations

import numpy as np

from .attention import sequence_rows, slot


def bits(masks, n):
    """[n][n]: whether drafted token i names drafted token k; without masks, k <= i."""
    if masks is None:
        return np.tril(np.ones((n, n), dtype=bool))
    named = np.zeros((n, n), dtype=bool)
    for i in range(n):
        for k in range(min(n, 64)):
            named[i, k] = (int(masks[i]) >> k) & 1
    return named


def seen_and_places(masks, n, length, window=0):
    """What each of a sequence's n drafted tokens sees [n][length], their places [n] and the positions' [length]."""
    base = length - n
    named = bits(masks, n)
    place = np.arange(length)
    here = np.array([base + (max(1, int(named[i].sum())) - 1 if masks is not None else i) for i in range(n)], dtype=int)
    seen = np.zeros((n, length), dtype=bool)
    for j in range(length):
        if j < base:
            seen[:, j] = True
        else:
            place[j] = here[j - base]
            seen[:, j] = named[:, j - base]
    if window:
        seen &= place[None, :] > here[:, None] - window
    return seen, here, place


def attention(q, k_cache, v_cache, table, q_starts, lengths, scale, masks=None, softcap=0.0, window=0, slopes=None):
    """(out [T][heads][dim], sum_j w_j |v_j|, largest sum |q k| over seen positions [T][heads]) in float64."""
    rows, heads, dim = q.shape
    kv_heads = k_cache.shape[1]
    out, mag, dots = np.zeros((rows, heads, dim)), np.zeros((rows, heads, dim)), np.zeros((rows, heads))
    for s in range(len(lengths)):
        a, b, length = int(q_starts[s]), int(q_starts[s + 1]), max(0, int(lengths[s]))
        if a == b:
            continue
        seen, here, place = seen_and_places(None if masks is None else masks[a:b], b - a, length, window)
        for h in range(heads):
            k, v, there = sequence_rows(k_cache, v_cache, table[s], length, h * kv_heads // heads)
            for t in range(a, b):
                at = np.flatnonzero(seen[t - a] & there)
                if len(at) == 0:
                    continue
                w = scale * (k[at] @ q[t, h].astype(np.float64))
                if softcap > 0:
                    w = softcap * np.tanh(w / softcap)
                if slopes is not None:
                    w = w + float(slopes[h]) * (place[at] - here[t - a])
                w = np.exp(w - w.max())
                w /= w.sum()
                out[t, h] = w @ v[at]
                mag[t, h] = w @ np.abs(v[at])
                dots[t, h] = (np.abs(k[at]) @ np.abs(q[t, h].astype(np.float64))).max()
    return out, mag, dots


def keep(k_cache, v_cache, table, starts, keep_starts, kept):
    """(k_cache, v_cache) after the move; v_cache may be None."""
    k, v = k_cache.copy(), None if v_cache is None else v_cache.copy()
    page, pages = (k_cache.shape[2] if v_cache is not None else k_cache.shape[1]), k_cache.shape[0]
    for s in range(len(starts)):
        for i, j in enumerate(kept[keep_starts[s]:keep_starts[s + 1]]):
            a, b = slot(table, s, int(starts[s]) + int(j), page, pages), slot(table, s, int(starts[s]) + i, page, pages)
            if a is None or b is None:
                continue
            if v is None:
                k[b[0], b[1]] = k_cache[a[0], a[1]]
            else:
                k[b[0], :, b[1]] = k_cache[a[0], :, a[1]]
                v[b[0], :, :, b[1]] = v_cache[a[0], :, :, a[1]]
    return k, v
