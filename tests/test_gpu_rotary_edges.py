"""GPU: rotary positions at the edges: every stride that keeps rows apart."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_279_gb300 as pkv
from paged_kv_cache_279_gb300 import _lib

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _clear_errors():
    pkv.read_device_errors(clear=True)
    yield
    assert pkv.read_device_errors(clear=True) == 0


def _rows(shape, dtype, seed):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape).astype(np.float32)).to(dtype)


@pytest.mark.parametrize("T,H", [(5, 4), (1, 4), (5, 1)])
def test_rows_apart_in_any_order(T, H):
    """Steps from token to token and head to head of either sign, one within the other or not: rows land where they belong,
    nothing else is written.  In place with the same strides too."""
    D, size, base = 64, 24000, 12000
    steps = (-704, -320, -256, -192, -128, -72, -64, -56, 0, 8, 56, 64, 72, 96, 128, 160, 192, 224, 256, 264, 320, 448, 1600)
    x, f = _rows((T, H, D), BF, 1).cuda(), pkv.rotary_frequencies(D, device="cuda")
    ps = torch.arange(T, dtype=torch.int32, device="cuda") * 77
    want = torch.empty_like(x)
    pkv.rotary_embed(want, x, ps, f)
    call, stream, met = _lib.load().rotary_embed, torch.cuda.current_stream().cuda_stream, 0
    for a in steps:
        for b in steps:
            at = a * torch.arange(T)[:, None] + b * torch.arange(H)[None]
            spots = at.flatten().sort().values
            if T * H > 1 and (spots[1:] - spots[:-1]).min() < D:
                continue
            met += 1
            where = (base + at[..., None] + torch.arange(D)).cuda()
            assert int(where.min()) >= 0 and int(where.max()) < size
            flat = torch.full((size,), 7.0, dtype=BF, device="cuda")
            clean = flat.clone()
            clean[where] = want
            p = flat.data_ptr() + 2 * base
            st = (ctypes.c_int64 * 4)(a, b, H * D, D)
            assert call(p, x.data_ptr(), ps.data_ptr(), f.data_ptr(), T, H, D, D, 0, st, 1.0, 0, pkv.PKV_BF16, stream) == pkv.PKV_OK
            assert torch.equal(flat, clean)
            flat.fill_(7.0)
            flat[where] = x
            st = (ctypes.c_int64 * 4)(a, b, a, b)
            assert call(p, p, ps.data_ptr(), f.data_ptr(), T, H, D, D, 0, st, 1.0, 0, pkv.PKV_BF16, stream) == pkv.PKV_OK
            assert torch.equal(flat, clean)
    assert met > 100
