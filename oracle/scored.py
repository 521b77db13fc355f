"""Oracle of scored attention: capped or biased scores, windows, documents and prefixes (test infrastructure).

Plain numpy float64 over contiguous per-sequence K/V, from the definition: the query at position p of a context of L
tokens scores the key at t with x = scale q.k, x = c tanh(x / c) (softcap c > 0), x = x - slope_h |p - t| (slopes given),
and sees it if t >= key_start and (t < prefix_len or (t <= p and (no window or p - t < window))).  No block table, no
tiles, no running maximum.  A query that sees nothing gets zeros.
"""
from __future__ import annotations

import numpy as np


def seen_keys(positions, length, window=0, prefix_len=0, key_starts=None):
    """Boolean [n, length]: which keys each of n queries sees."""
    p = np.asarray(positions, dtype=np.int64)[:, None]
    t = np.arange(length, dtype=np.int64)[None, :]
    behind = t <= p
    if window:
        behind &= p - t < window
    seen = behind | (t < prefix_len)
    if key_starts is not None:
        seen &= t >= np.asarray(key_starts, dtype=np.int64)[:, None]
    return seen


def scored_attention(q, k, v, scale, softcap=0.0, slopes=None, window=0, prefix_len=0, key_starts=None):
    """One sequence: q [n, Hq, D] at the last n positions of a context k, v [L, Hkv, D] -> (out [n, Hq, D], and
    sum_t w_t |v_t| of the same shape, the size against which weights' roundings count)."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    n, Hq, D = q.shape
    L, Hkv = k.shape[0], k.shape[1]
    out, size = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    if n == 0 or L == 0:
        return out, size
    p = np.arange(L - n, L, dtype=np.int64)
    seen = seen_keys(p, L, window, prefix_len, key_starts)
    away = np.abs(p[:, None] - np.arange(L)[None, :]).astype(np.float64)
    for h in range(Hq):
        g = h // (Hq // Hkv)
        x = scale * (q[:, h] @ k[:, g].T)
        if softcap > 0:
            x = softcap * np.tanh(x / softcap)
        if slopes is not None:
            x = x - float(slopes[h]) * away
        x = np.where(seen, x, -np.inf)
        top = x.max(axis=1, keepdims=True)
        w = np.exp(x - np.where(np.isfinite(top), top, 0.0))
        total = w.sum(axis=1, keepdims=True)
        w = w / np.where(total > 0, total, 1.0)
        out[:, h] = w @ v[:, g]
        size[:, h] = w @ np.abs(v[:, g])
    return out, size
