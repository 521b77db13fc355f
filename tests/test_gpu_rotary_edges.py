"""GPU: rotary positions at the edges: every stride that keeps rows apart, attention over what was written, large frequencies."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_279_gb300 as pkv
from oracle import rotary
from paged_kv_cache_279_gb300 import _lib

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


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


@pytest.mark.parametrize("T,Hq,Hkv,D,B", [(50, 8, 2, 64, 16), (77, 4, 4, 128, 32)])
def test_attention_over_rows_that_were_rotated_and_written(T, Hq, Hkv, D, B):
    """kv_cache_write_rotary stores what rotary_embed and kv_cache_write do, bit for bit; the attention calls read it, queries
    and all: within the errors of their own arithmetic on the stored numbers (scores of D products and exponentials in
    float32, weights and the output rounded to bf16)."""
    from oracle.multi_token import multi_token_attention
    qkv = _rows((T, Hq + 2 * Hkv, D), BF, 8).cuda()
    f, at = pkv.rotary_frequencies(D, device="cuda"), torch.arange(T, device="cuda")
    tables = torch.tensor([[5, 2, 7, 0]], dtype=torch.int32, device="cuda")
    slots = tables[0].long()[at // B] * B + at % B
    kc, vc, kc2, vc2 = (torch.full((8, Hkv, B, D), float("nan"), dtype=BF, device="cuda") for _ in range(4))
    q, q2 = (torch.empty((T, Hq, D), dtype=BF, device="cuda") for _ in range(2))
    k, v = qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    pkv.kv_cache_write_rotary(k, v, kc, vc, slots, at.int(), f, q=qkv[:, :Hq], q_out=q)
    rot = torch.empty((T, Hkv, D), dtype=BF, device="cuda")
    pkv.rotary_embed(rot, k, at.int(), f)
    pkv.rotary_embed(q2, qkv[:, :Hq], at.int(), f)
    pkv.kv_cache_write(rot, v.contiguous(), kc2, vc2, slots)
    bits = lambda x: x.view(torch.int16)  # noqa: E731  (NaN in unused slots)
    assert torch.equal(q, q2) and torch.equal(bits(kc), bits(kc2)) and torch.equal(bits(vc), bits(vc2))
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    out, one = torch.empty_like(q), torch.empty((1, Hq, D), dtype=BF, device="cuda")
    pkv.paged_attention_multi_token(out, q, kc, vc, tables, lens, torch.tensor([0, T], dtype=torch.int32, device="cuda"), 0.125, T, T)
    pkv.paged_attention_decode(one, q[-1:].contiguous(), kc, vc, tables, lens, 0.125, T)
    qd, kd, vd = (x.double().cpu().numpy() for x in (q, rot, v))
    ref, = multi_token_attention([qd], [kd], [vd], 0.125)
    spread, = multi_token_attention([qd], [kd], [np.abs(vd)], 0.125)
    g = Hq // Hkv
    reach = 0.125 * max((np.abs(qd[:, h]) @ np.abs(kd[:, h // g]).T).max() for h in range(Hq))
    rel = 2 * (reach * (D + 4) * 2.0 ** -24 + 2.0 ** -21 + (T + 2) * 2.0 ** -24) + 2 * 2.0 ** -8
    tol = rel * spread + 2.0 ** -8 * np.abs(ref)
    assert np.all(np.abs(out.double().cpu().numpy() - ref) <= tol)
    assert np.all(np.abs(one.double().cpu().numpy()[0] - ref[-1]) <= tol[-1])


def test_large_frequencies():
    """Angles within |p| (2^-64 + |f| 2^-72) turns, then the roundings of float32 (2^-21 of the pair)."""
    pos = np.array([1, -1, 1000, -77777, 10 ** 6, 2 ** 31 - 1, -2 ** 31], dtype=np.int64)
    f = np.array([1e3, 1e6, 2.0 ** 30 + 0.1, 1e9, -1e10, 1e11, 1e12, 3e5])
    x = _rows((len(pos), 3, 16), F32, 5)
    out = torch.empty_like(x, device="cuda")
    pkv.rotary_embed(out, x.cuda(), torch.from_numpy(pos).int().cuda(), torch.from_numpy(f).cuda())
    x64 = x.double().numpy()
    want = rotary.rotate(x64, pos, f, far=True)
    angle = 2 * np.pi * np.abs(pos)[:, None] * (2.0 ** -64 + np.abs(f) * 2.0 ** -72)
    pair = np.abs(x64[..., :8]) + np.abs(x64[..., 8:])
    tol = np.concatenate([(2.0 ** -21 + angle)[:, None] * pair] * 2, -1)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= tol)
    assert np.median(tol / (np.abs(want) + 1e-30)) < 1e-5  # (most of these angles are as good as exact)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_read_more_than_once(dtype):
    """One row for all heads or all tokens (steps of 0 where rows are read), and slots of no token."""
    T, H, D, B = 7, 5, 64, 16
    f, ps = pkv.rotary_frequencies(D, device="cuda"), torch.arange(T, dtype=torch.int32, device="cuda") * 9
    for x in (_rows((T, 1, D), dtype, 1).cuda().expand(T, H, D), _rows((1, H, D), dtype, 2).cuda().expand(T, H, D)):
        want, out = torch.empty((T, H, D), dtype=dtype, device="cuda"), torch.empty((T, H, D), dtype=dtype, device="cuda")
        pkv.rotary_embed(want, x.contiguous(), ps, f)
        assert torch.equal(pkv.rotary_embed(out, x, ps, f), want)
        kc, vc = torch.full((2, H, B, D), 7.0, dtype=dtype, device="cuda"), torch.full((2, H, B, D), 7.0, dtype=dtype, device="cuda")
        slots = torch.tensor([3, -1, 17, 0, 31, -5, 16], device="cuda")
        pkv.kv_cache_write_rotary(x, x, kc, vc, slots, ps, f)
        for t, s in enumerate(slots.tolist()):
            if s >= 0:
                assert torch.equal(kc[s // B, :, s % B], want[t]) and torch.equal(vc[s // B, :, s % B], x[t])
        assert int((kc == 7.0).all(-1).sum()) == H * (2 * B - 5)
