"""Limits of the latent attention and rotary calls that are refused on the host (no GPU)."""
import ctypes

import pytest

import paged_kv_cache_279_gb300 as pkv
from paged_kv_cache_279_gb300 import _lib

P = ctypes.c_void_p(256)  # aligned, never dereferenced


@pytest.mark.parametrize("S", [2 ** 31 - 1, 0x7ffff001])
@pytest.mark.parametrize("dt", [pkv.PKV_F32, pkv.PKV_BF16])
def test_sequences_past_31_bits(S, dt):
    """Indices of sequences are 32-bit sums with the threads or blocks of a launch."""
    f = _lib.load().paged_latent_attention_multi_token
    assert f(P, P, P, P, P, P, S, 10, 16, 512, 16, 4, 16, 5, 64, 0.1, P, 1 << 40, dt, None) == pkv.PKV_ERR_UNSUPPORTED


X, Y = P, ctypes.c_void_p(1 << 20)  # two tensors


def _str(*s):
    return (ctypes.c_int64 * len(s))(*s)


def _embed(out, x, st, T, H, D):
    return _lib.load().rotary_embed(out, x, P, P, T, H, D, D, 0, _str(*st), 1.0, 0, pkv.PKV_BF16, None)


def _write(out, x, st, T, H, D):
    return _lib.load().kv_cache_write_rotary(out, x, P, P, P, P, P, P, P, T, H, 2, D, D, 0, 16, 64, _str(*st, 2 * D, D, 2 * D, D), 1.0, 0,
                                             pkv.PKV_BF16, None)


def _latent(out, x, st, T, H, D):
    return _lib.load().latent_cache_write(out, x, P, P, P, P, P, P, T, H, 512, 16, 64, _str(*st, 576, 576), 1.0, 0, pkv.PKV_BF16, None)


CALLS = [_embed, _write, _latent]


def _apart(st, T, H, D):
    spots = sorted(t * st[0] + h * st[1] for t in range(T) for h in range(H))
    return all(b - a >= D for a, b in zip(spots, spots[1:]))


@pytest.mark.parametrize("call", CALLS)
def test_written_rows_that_overlap(call):
    T, H, D = 5, 4, 64
    read = (1 << 20, 64)
    steps = (-704, -320, -256, -192, -128, -72, -64, -56, -8, 0, 8, 56, 64, 72, 96, 128, 160, 192, 224, 256, 264, 320, 448, 1600)
    bad = [(a, b) for a in steps for b in steps if not _apart((a, b), T, H, D)]
    assert len(bad) > 100
    for st in bad:
        assert call(X, Y, st + read, T, H, D) == pkv.PKV_ERR_INVALID, st
    assert call(X, Y, (0, 56) + read, 1, H, D) == pkv.PKV_ERR_INVALID and call(X, Y, (56, 0) + read, T, 1, D) == pkv.PKV_ERR_INVALID
    assert call(X, Y, (1 << 56, -(1 << 56) + 56) + read, 3, 3, D) == pkv.PKV_ERR_INVALID


@pytest.mark.parametrize("call", CALLS)
def test_in_place_with_other_strides(call):
    for st in ((512, 64, 256, 64), (256, 64, 512, 64), (1024, 128, 1024, 64), (64, 320, 256, 64)):
        assert call(X, X, st, 5, 4, 64) == pkv.PKV_ERR_INVALID


def test_frequencies_past_float64():
    """Rotation takes an infinite or NaN frequency for 0: none is handed out."""
    f, out = _lib.load().rotary_frequencies, (ctypes.c_double * 4)()
    assert f(out, 8, 1e-300, 1e-60, 0.0, 1.0, 32.0) == pkv.PKV_OK and out[3] == pytest.approx(1e285, rel=1e-9)
    assert f(out, 8, 1e-300, 1e-100, 0.0, 1.0, 32.0) == pkv.PKV_ERR_INVALID              # infinite
    assert f(out, 8, 1e-300, 4.0, 1e200, -1e308, 1e308) == pkv.PKV_ERR_INVALID           # infinity over infinity
    with pytest.raises(pkv.PkvError):
        pkv.rotary_frequencies(8, base=1e-300, factor=1e-100)
