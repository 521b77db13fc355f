"""Rotation of rows by their positions, and the frequencies of its pairs.

TEST INFRASTRUCTURE ONLY (same rule as the rest of ``oracle/``).

No page describes it: it is the usual definition, with the two layouts of pairs
that models use.  Rows x [T, H, D] at positions p [T]; the entries from
``offset`` on, R = 2 len(freqs) of them, form pairs, pair i = (x1, x2):
    y1 = x1 c - x2 s,  y2 = x2 c + x1 s,  c = a cos(p f_i),  s = a sin(p f_i)
"""
from __future__ import annotations

from decimal import Decimal, localcontext

import numpy as np

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


def angle(p: int, f: float) -> float:
    """p f modulo a turn, in [-pi, pi], correct to float64 for any integer p and float64 f."""
    with localcontext() as ctx:
        ctx.prec = 75
        turns = Decimal(int(p)) * Decimal(float(f)) / (2 * PI)
        turns -= turns.to_integral_value()
        return float(turns * 2 * PI)


def rotate(x, positions, freqs, amplitude=1.0, interleaved=False, offset=0, far=False):
    """float64 rows; ``far``: angles by ``angle`` (positions for which p f loses digits in float64)."""
    y = np.array(x, dtype=np.float64)
    n = len(freqs)
    if far:
        ang = np.array([[angle(p, f) for f in freqs] for p in positions])
    else:
        ang = np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(freqs, dtype=np.float64)
    c, s = (amplitude * g(ang)[:, None, :] for g in (np.cos, np.sin))
    i1 = offset + (2 * np.arange(n) if interleaved else np.arange(n))
    i2 = i1 + (1 if interleaved else n)
    x1, x2 = y[..., i1].copy(), y[..., i2].copy()
    y[..., i1], y[..., i2] = x1 * c - x2 * s, x2 * c + x1 * s
    return y


def frequencies(rotary_dim, base=10000.0, factor=1.0, original_len=0.0, low_turns=1.0, high_turns=32.0):
    out = []
    for i in range(rotary_dim // 2):
        f = base ** (-2.0 * i / rotary_dim)
        keep = 0.0
        if original_len:
            turns = original_len * f / (2.0 * np.pi)
            keep = min(max((turns - low_turns) / (high_turns - low_turns), 0.0), 1.0)
        out.append(keep * f + (1.0 - keep) * f / factor)
    return np.array(out)
