"""Head norm, rotary position, paged cache and attention in float64, one token
and one head at a time (the definitions of q4g128_rope_append,
q4g128_attn_decode and q4g128_attn_prefill in include/q4g128.h).
"""
from __future__ import annotations

import numpy as np


def rotated(x, position, inv_freq, rot, interleaved=False, mscale=1.0, weight=None, eps=1e-6):
    """One head's row x [dim] after norm and rotation."""
    x = np.asarray(x, dtype=np.float64).copy()
    if weight is not None:
        x = x / np.sqrt(np.mean(x * x) + eps) * np.asarray(weight, dtype=np.float64)
    y = x.copy()
    for i in range(rot // 2):
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        a = float(position) * float(inv_freq[i])
        c, s = np.cos(a), np.sin(a)
        y[lo] = mscale * (x[lo] * c - x[hi] * s)
        y[hi] = mscale * (x[hi] * c + x[lo] * s)
    return y


def slot(table, sequence, position, page, pages):
    """(page number, offset) of a position, or None when it has no place in the cache."""
    if not 0 <= sequence < table.shape[0] or position < 0 or position // page >= table.shape[1]:
        return None
    p = int(table[sequence, position // page])
    return (p, position % page) if 0 <= p < pages else None


def sequence_rows(k_cache, v_cache, table_row, length, kv_head):
    """K and V [length][dim] of one sequence and kv head in float64, and which positions have a page."""
    pages, _, page, dim = k_cache.shape
    k, v = np.zeros((length, dim)), np.zeros((length, dim))
    there = np.zeros(length, dtype=bool)
    for j in range(length):
        p = int(table_row[j // page])
        if 0 <= p < pages:
            there[j] = True
            k[j] = k_cache[p, kv_head, j % page]
            v[j] = v_cache[p, kv_head, :, j % page]
    return k, v, there


def weights(q, k, position, seen, scale, softcap=0.0, slope=0.0):
    """Softmax weights [length] of one query over the positions in `seen` (all zero if there is none)."""
    w = np.zeros(len(k))
    at = np.flatnonzero(seen)
    if len(at) == 0:
        return w
    s = scale * (k[at] @ np.asarray(q, dtype=np.float64))
    if softcap > 0:
        s = softcap * np.tanh(s / softcap)
    s = s + slope * (at - position)
    e = np.exp(s - s.max())
    w[at] = e / e.sum()
    return w


def visible(length, position, there, window=0, prefix=0):
    j = np.arange(length)
    seen = j <= position
    if window:
        seen &= j > position - window
    if position >= 0:
        seen |= j < prefix
    return seen & there


def attention(q, k_cache, v_cache, table, q_starts, lengths, scale, softcap=0.0, window=0, slopes=None, prefix=None):
    """(out [T][heads][dim], magnitude sum_j w_j |v_j|, largest sum |q k| over seen positions [T][heads]) in float64."""
    rows, heads, dim = q.shape
    kv_heads = k_cache.shape[1]
    out, mag, dots = np.zeros((rows, heads, dim)), np.zeros((rows, heads, dim)), np.zeros((rows, heads))
    for s in range(len(lengths)):
        a, b, n = int(q_starts[s]), int(q_starts[s + 1]), max(0, int(lengths[s]))
        for h in range(heads):
            k, v, there = sequence_rows(k_cache, v_cache, table[s], n, h * kv_heads // heads)
            for t in range(a, b):
                position = n - (b - t)
                seen = visible(n, position, there, window, 0 if prefix is None else int(prefix[s]))
                w = weights(q[t, h], k, position, seen, scale, softcap, 0.0 if slopes is None else float(slopes[h]))
                at = np.flatnonzero(seen)
                if len(at):
                    out[t, h] = w[at] @ v[at]
                    mag[t, h] = w[at] @ np.abs(v[at])
                    dots[t, h] = (np.abs(k[at]) @ np.abs(q[t, h].astype(np.float64))).max()
    return out, mag, dots
