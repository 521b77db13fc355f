"""paged_attention_decode_scored with new tokens: a call that is refused is refused before it stores them (no GPU: a store
that went first would come back as a CUDA error, there being no device)."""
import ctypes

import pytest
import torch

import paged_kv_cache_279_gb300 as pkv
from paged_kv_cache_279_gb300 import _lib

P = ctypes.c_void_p(256)  # aligned, never dereferenced


def call(ws=P, nws=1 << 40, S=2, Hq=8, Hkv=8, maxB=10000, maxL=100000, dt=1, window=0):
    return _lib.load().paged_attention_decode_scored(P, P, P, P, P, P, P, P, S, Hq, Hkv, 128, 16, maxB, 16, maxL, 0.1, 0.0, None,
                                                     window, None, None, ws, nws, dt, None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the accepted call would run on made-up addresses")
@pytest.mark.parametrize("dt", [0, 1])
def test_refused_before_the_store(dt):
    assert call(None, 0, dt=dt) == pkv.PKV_ERR_INVALID                      # no workspace
    assert call(nws=100, dt=dt) == pkv.PKV_ERR_INVALID                      # too small a one
    assert call(ctypes.c_void_p(256 + 16), dt=dt) == pkv.PKV_ERR_INVALID    # not aligned
    assert call(window=-1, dt=dt) == pkv.PKV_ERR_INVALID
    # more KV heads than a grid, or a single sequence's tiles, hold
    assert call(Hq=1 << 17, Hkv=1 << 17, maxB=1 << 24, maxL=1 << 28, dt=dt) == pkv.PKV_ERR_UNSUPPORTED
    assert call(dt=dt) == pkv.PKV_ERR_CUDA                                  # valid, but for the device
