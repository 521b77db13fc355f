"""The scored attention and row-scaled FP8 calls refuse bad arguments on the host, before any device work (no GPU)."""
import ctypes

import pytest

import paged_kv_cache_279_gb300 as pkv
from paged_kv_cache_279_gb300 import _lib

P = ctypes.c_void_p(256)  # aligned, never dereferenced: each call below is refused before a launch


@pytest.mark.parametrize("name", ["kv_cache_write_fp8_rows", "kv_cache_read_fp8_rows"])
def test_rows_calls(name):
    f = getattr(_lib.load(), name)

    def call(p=None, T=4, Hkv=8, D=128, B=16, NB=64, dt=1):
        return f(p, p, p, p, p, p, p, T, Hkv, D, B, NB, dt, None)
    assert call() == pkv.PKV_ERR_INVALID
    assert call(P, D=96) == pkv.PKV_ERR_UNSUPPORTED
    assert call(P, B=8) == pkv.PKV_ERR_UNSUPPORTED
    assert call(P, dt=2) == pkv.PKV_ERR_UNSUPPORTED
    assert call(P, T=-1) == pkv.PKV_ERR_INVALID
    assert call(P, Hkv=0) == pkv.PKV_ERR_INVALID
    assert call(P, NB=0) == pkv.PKV_ERR_INVALID
    assert call(ctypes.c_void_p(264)) == pkv.PKV_ERR_INVALID
    assert call(T=0) == pkv.PKV_OK
    assert call(P, T=2 ** 31 - 1, Hkv=1 << 20) == pkv.PKV_ERR_UNSUPPORTED  # more rows than a grid holds


def _decode(p=None, knew=None, vnew=None, S=2, Hq=32, Hkv=8, D=128, B=16, maxB=4, NB=16, maxL=64, scale=0.1, cap=0.0,
            window=0, ws=None, nws=0, dt=1):
    return _lib.load().paged_attention_decode_scored(p, p, knew, vnew, p, p, p, p, S, Hq, Hkv, D, B, maxB, NB, maxL, scale,
                                                     cap, None, window, None, None, ws, nws, dt, None)


def _rows(p=None, S=2, Hq=32, Hkv=8, D=128, B=16, maxB=4, NB=16, maxL=64, scale=0.1, cap=0.0, window=0, ws=None, nws=0):
    return _lib.load().paged_attention_decode_scored_fp8_rows(p, p, p, p, p, p, p, p, S, Hq, Hkv, D, B, maxB, NB, maxL, scale,
                                                              cap, None, window, None, None, ws, nws, None)


def _multi(p=None, S=2, T=10, Hq=32, Hkv=8, D=128, B=16, maxB=4, NB=16, maxQ=5, maxL=64, scale=0.1, cap=0.0, window=0,
           ws=None, nws=0):
    return _lib.load().paged_attention_multi_token_scored(p, p, p, p, p, p, p, S, T, Hq, Hkv, D, B, maxB, NB, maxQ, maxL,
                                                          scale, cap, None, window, None, None, ws, nws, None)


@pytest.mark.parametrize("call", [_decode, _rows, _multi])
def test_attention_calls(call):
    assert call() == pkv.PKV_ERR_INVALID                       # null pointers
    assert call(P, Hq=30) == pkv.PKV_ERR_INVALID
    assert call(P, Hq=72) == pkv.PKV_ERR_UNSUPPORTED           # 9 query heads per KV head
    assert call(P, D=96) == pkv.PKV_ERR_UNSUPPORTED
    assert call(P, B=12) == pkv.PKV_ERR_UNSUPPORTED
    assert call(P, S=-1) == pkv.PKV_ERR_INVALID
    assert call(P, maxB=0) == pkv.PKV_ERR_INVALID
    assert call(P, maxL=-1) == pkv.PKV_ERR_INVALID
    assert call(P, window=-1) == pkv.PKV_ERR_INVALID
    for bad in (float("nan"), float("inf"), -1.0):
        assert call(P, cap=bad) == pkv.PKV_ERR_INVALID
    assert call(P, scale=float("nan")) == pkv.PKV_ERR_INVALID
    assert call(P, scale=float("inf")) == pkv.PKV_ERR_INVALID
    assert call(ctypes.c_void_p(264)) == pkv.PKV_ERR_INVALID   # not 16-byte aligned
    assert call(P, maxB=1 << 28) == pkv.PKV_ERR_INVALID        # positions past 31 bits
    assert call(P, NB=1 << 28) == pkv.PKV_ERR_UNSUPPORTED      # cache rows past 31 bits
    assert call(P, maxL=100000, maxB=10000) == pkv.PKV_ERR_INVALID   # no workspace
    assert call(P, maxL=100000, maxB=10000, ws=ctypes.c_void_p(256 + 16), nws=1 << 40) == pkv.PKV_ERR_INVALID
    assert call(P, maxL=100000, maxB=10000, ws=P, nws=100) == pkv.PKV_ERR_INVALID
    assert call(S=0) == pkv.PKV_OK


def test_only_their_own():
    assert _rows(P, B=8) == pkv.PKV_ERR_UNSUPPORTED
    assert _decode(P, dt=2) == pkv.PKV_ERR_UNSUPPORTED
    assert _decode(P, knew=P) == pkv.PKV_ERR_INVALID           # K without V
    assert _decode(P, knew=P, vnew=P, maxL=0) == pkv.PKV_ERR_INVALID
    assert _multi(P, maxQ=0) == pkv.PKV_ERR_INVALID
    assert _multi(P, T=-1) == pkv.PKV_ERR_INVALID
    assert _multi(T=0) == pkv.PKV_OK


def test_workspace_sizes():
    lib = _lib.load()
    d, m = lib.paged_attention_decode_scored_workspace_size, lib.paged_attention_multi_token_scored_workspace_size
    for f in (d, m):
        assert f(0, 32, 128, 100) == 0 and f(4, 0, 128, 100) == 0 and f(4, 32, 0, 100) == 0 and f(4, 32, 128, 0) == 0
        assert f(4, 32, 128, 100000) > 0 and f(4, 32, 128, 100000) % 256 == 0
