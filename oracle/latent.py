"""Latent rows, their attention (absorbed form) and the keys and values expanded
from them, in float64 (the definitions of the q4g128_latent calls in
include/q4g128.h), one token and one head at a time.
"""
from __future__ import annotations

import numpy as np

from .attention import rotated, slot
from .drafts import seen_and_places

ROT = 64


def row(x, position, inv_freq, latent, interleaved=False, mscale=1.0, norm=None, eps=1e-6):
    """One token's cache row [latent + 64] of its projection x."""
    x = np.asarray(x, dtype=np.float64)
    body = x[:latent]
    if norm is not None:
        body = body / np.sqrt(np.mean(body * body) + eps) * np.asarray(norm, dtype=np.float64)
    return np.concatenate([body, turned(x[latent:latent + ROT], position, inv_freq, interleaved, mscale)])


def turned(x, position, inv_freq, interleaved=False, mscale=1.0):
    return np.asarray(x, dtype=np.float64) if inv_freq is None else rotated(x, position, inv_freq, ROT, interleaved, mscale)


def rows_of(cache, table_row, length):
    """Cached rows [length][latent + 64] of a sequence in float64, and which positions have a page."""
    pages, page, dim = cache.shape
    rows, there = np.zeros((length, dim)), np.zeros(length, dtype=bool)
    for j in range(length):
        p = int(table_row[j // page])
        if 0 <= p < pages:
            there[j], rows[j] = True, cache[p, j % page]
    return rows, there


def attention(q, cache, table, q_starts, lengths, scale, masks=None):
    """(out [T][heads][latent], sum_j w_j |c_j|, largest sum |q c| over seen positions [T][heads]) in float64."""
    tokens, heads, dim = q.shape
    latent = dim - ROT
    out, mag, dots = np.zeros((tokens, heads, latent)), np.zeros((tokens, heads, latent)), np.zeros((tokens, heads))
    for s in range(len(lengths)):
        a, b, length = int(q_starts[s]), int(q_starts[s + 1]), max(0, int(lengths[s]))
        if a == b:
            continue
        seen, _, _ = seen_and_places(None if masks is None else masks[a:b], b - a, length)
        rows, there = rows_of(cache, table[s], length)
        for t in range(a, b):
            at = np.flatnonzero(seen[t - a] & there)
            if len(at) == 0:
                continue
            x = q[t].astype(np.float64)
            w = scale * (x @ rows[at].T)
            w = np.exp(w - w.max(-1, keepdims=True))
            w /= w.sum(-1, keepdims=True)
            out[t], mag[t] = w @ rows[at, :latent], w @ np.abs(rows[at, :latent])
            dots[t] = (np.abs(x) @ np.abs(rows[at]).T).max(-1)
    return out, mag, dots


def expanded(cache, table, lengths, weights, heads):
    """Keys [S][length][heads][value + 64] and values [S][length][heads][value] of every position, float64.

    weights [heads * 2 value][latent]: the heads' key rows, then their value rows, as they enter the product.
    """
    latent = cache.shape[2] - ROT
    value = weights.shape[0] // heads // 2
    w = np.asarray(weights, dtype=np.float64).reshape(heads, 2, value, latent)
    keys, values = [], []
    for s in range(len(lengths)):
        rows, _ = rows_of(cache, table[s], max(0, int(lengths[s])))
        k = np.einsum("jl,hvl->jhv", rows[:, :latent], w[:, 0])
        keys.append(np.concatenate([k, np.broadcast_to(rows[:, None, latent:], (len(rows), heads, ROT))], -1))
        values.append(np.einsum("jl,hvl->jhv", rows[:, :latent], w[:, 1]))
    return keys, values


__all__ = ["ROT", "row", "turned", "rows_of", "attention", "expanded", "slot"]
