"""Attention over one latent row a token, shared by all heads (absorbed form).

TEST INFRASTRUCTURE ONLY (same rule as the rest of ``oracle/``).

No page describes it.  Rows c_t = [latent_t | key part_t] of a context in order;
the query at position p, every head h:
    out[h] = sum_{t <= p} softmax_t(scale q[h] . c_t) latent_t
"""
from __future__ import annotations

import numpy as np


def latent_attention(q_seqs, rows_seqs, scale, latent):
    """fp64 causal attention of each sequence's last Q_s positions: q_seqs[s] [Q_s, H, D], rows_seqs[s] [L_s, D].

    Returns [(out, spread, reach)]: out and spread = sum_t w_t |latent_t| [Q_s, H, latent], reach = the largest
    scale * sum_i |q_i c_i| of the query's visible tokens [Q_s, H, 1]: what rounding errors are proportional to.
    A query that sees nothing gets zeros."""
    res = []
    for q, rows in zip(q_seqs, rows_seqs):
        q, rows = np.asarray(q, dtype=np.float64), np.asarray(rows, dtype=np.float64)
        n, H, D = q.shape
        L = rows.shape[0]
        out, spread, reach = np.zeros((n, H, latent)), np.zeros((n, H, latent)), np.zeros((n, H, 1))
        for i in range(n):
            p = L - n + i
            if p < 0:
                continue
            c = rows[:p + 1]
            x = scale * (q[i] @ c.T)
            w = np.exp(x - x.max(-1, keepdims=True))
            w /= w.sum(-1, keepdims=True)
            out[i], spread[i] = w @ c[:, :latent], w @ np.abs(c[:, :latent])
            reach[i] = (abs(scale) * (np.abs(q[i]) @ np.abs(c).T)).max(-1, keepdims=True)
        res.append((out, spread, reach))
    return res
