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
