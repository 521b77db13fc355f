"""Oracle of the row-scaled FP8 cache (test infrastructure): E4M3 codes and one power-of-two scale per row.

Numpy float64 from the format's definition, element by element, apart from the codes' table and rounding, which are those
of oracle/fp8_e4m3.py: e is the smallest integer with max |x| <= 448 * 2^e over the finite entries, held in [-100, 120];
code = e4m3(x * 2^-e); value = e4m3(code) * 2^e.
"""
from __future__ import annotations

import numpy as np

from . import fp8_e4m3


def row_exponent(x):
    """e of rows x [..., D], int64 [...]."""
    x = np.asarray(x, dtype=np.float64)
    a = np.where(np.isfinite(x), np.abs(x), 0.0).max(axis=-1)
    e = np.full(a.shape, -100, dtype=np.int64)
    for i in np.ndindex(a.shape):
        k = -100
        while k < 120 and a[i] > 448.0 * 2.0 ** k:
            k += 1
        e[i] = k
    return e


def quantise_rows(x):
    """(codes uint8 [..., D], scale bytes uint8 [...])."""
    x = np.asarray(x, dtype=np.float64)
    e = row_exponent(x)
    return fp8_e4m3.float_to_e4m3(x * np.exp2(-e.astype(np.float64))[..., None]), (e + 127).astype(np.uint8)


def row_values(codes, scale_bytes):
    return fp8_e4m3.e4m3_to_float(codes) * np.exp2(np.asarray(scale_bytes, dtype=np.float64) - 127.0)[..., None]
