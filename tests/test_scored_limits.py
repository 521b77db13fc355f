"""Shapes at the ends of the integers are refused by the scored calls, whatever their products come to (no GPU)."""
import ctypes

import pytest

import paged_kv_cache_279_gb300 as pkv
from paged_kv_cache_279_gb300 import _lib

P = ctypes.c_void_p(256)  # aligned, never dereferenced: each call below is refused before a launch
BIG = 1 << 62


@pytest.mark.parametrize("Hkv", [1 << 20, 1 << 26, 123456789 >> 1])
@pytest.mark.parametrize("maxL", [1 << 30, (1 << 30) - 383, 2 ** 31 - 1])
def test_products_of_maxima(Hkv, maxL):
    lib, maxB = _lib.load(), 1 << 27
    for T in (2 ** 31 - 1, (1 << 30) + 1):
        assert lib.paged_attention_multi_token_scored(P, P, P, P, P, P, P, 2 ** 31 - 1, T, Hkv, Hkv, 128, 8, maxB, 1, 2 ** 31 - 1,
                                                      maxL, 0.1, 0.0, None, 0, None, None, P, BIG, None) == pkv.PKV_ERR_UNSUPPORTED
    assert lib.paged_attention_decode_scored(P, P, P, P, P, P, P, P, 2 ** 31 - 1, Hkv, Hkv, 128, 8, maxB, 1, maxL, 0.1, 0.0, None, 0,
                                             None, None, P, BIG, 1, None) == pkv.PKV_ERR_UNSUPPORTED


def test_a_workspace_past_64_bits():
    lib = _lib.load()
    for S in (2 ** 31 - 1, 1 << 30):
        for L in ((1 << 25) - 512, 3 << 23):
            for H in (1 << 18, 65535 * 8):
                assert lib.paged_attention_decode_scored_workspace_size_for(S, H, 128, L, 0) > BIG
                assert lib.paged_attention_decode_scored(P, P, P, P, P, P, P, P, S, H, H // 8, 128, 8, 1 << 20, 1, L, 0.1, 0.0, None,
                                                         0, None, None, P, BIG, 0, None) == pkv.PKV_ERR_INVALID
