"""GPU: rotary positions alone and on the way into the paged caches, against the oracle."""
import numpy as np
import pytest
import torch

import paged_kv_cache_279_gb300 as pkv
from oracle import rotary

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _clear_errors():
    pkv.read_device_errors(clear=True)
    yield


def _rows(shape, dtype, seed):
    r = np.random.default_rng(seed)
    return torch.from_numpy(r.standard_normal(shape).astype(np.float32)).to(dtype)


def _check(got, x, positions, freqs, dtype, amplitude=1.0, interleaved=False, offset=0, far=False):
    """Copied entries bit for bit; rotated ones within the roundings of float32: c and s off by at most a (2^-23 for
    sincospif, 2^-23.3 for the angle, 2^-24 for the factor a), two products and a sum (2^-24 each), in all less than
    2^-21 a (|x1| + |x2|), and one rounding to the rows' type."""
    R = 2 * len(freqs)
    got, x64 = got.double().cpu().numpy(), x.double().cpu().numpy()
    want = rotary.rotate(x64, positions, freqs, amplitude, interleaved, offset, far)
    assert np.array_equal(got[..., :offset], x64[..., :offset]) and np.array_equal(got[..., offset + R:], x64[..., offset + R:])
    part = np.abs(x64[..., offset:offset + R])
    pair = part.reshape(part.shape[:-1] + ((R // 2, 2) if interleaved else (2, R // 2))).sum(-1 if interleaved else -2)
    size = np.repeat(pair, 2, -1) if interleaved else np.concatenate([pair, pair], -1)
    w = want[..., offset:offset + R]
    tol = abs(amplitude) * size * 2.0 ** -21 + (np.abs(w) * torch.finfo(dtype).eps / 2 if dtype == BF else 0.0)
    assert np.all(np.abs(got[..., offset:offset + R] - w) <= tol)


SHAPES = [(1, 1, 64, 64, 0), (1, 64, 128, 128, 0), (3, 5, 128, 64, 0), (7, 3, 64, 16, 48), (33, 40, 128, 96, 32), (2, 7, 48, 32, 16),
          (300, 8, 128, 128, 0), (5, 2, 576, 64, 512), (9, 1, 256, 256, 0), (12000, 2, 64, 32, 0)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,D,R,off", SHAPES)
def test_embed(dtype, interleaved, T, H, D, R, off):
    x = _rows((T, H, D), dtype, T + R)
    f = pkv.rotary_frequencies(R, factor=4.0, original_len=100.0)
    pos = np.random.default_rng(1).integers(0, 200000, T)
    dev = x.cuda()
    out = torch.full_like(dev, 7.0)
    args = (torch.from_numpy(pos).int().cuda(), f.cuda())
    kw = dict(amplitude=1.25, interleaved=interleaved, offset=off)
    assert pkv.rotary_embed(out, dev, *args, **kw) is out
    _check(out, x, pos, f.numpy(), dtype, 1.25, interleaved, off)
    pkv.rotary_embed(dev, dev, *args, **kw)  # in place: the same bits
    assert torch.equal(dev, out)


def test_far_and_negative_positions():
    pos = np.array([0, 1, -1, -77, 10 ** 6, 10 ** 8 + 7, 2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1], dtype=np.int64)
    f = np.array([1.0, 0.1, 1e-3, 1e-9, 3.7, -0.5, 1e5, 2.0 ** -60, 0.0, 2 * np.pi, 1e-300, 6.0, 0.7, 1e3, 1e-5, 12345.678])
    x = _rows((len(pos), 2, 32), F32, 3)
    x[:, 1, 16:] = 0.0  # sines alone: their relative precision
    out = torch.empty_like(x, device="cuda")
    pkv.rotary_embed(out, x.cuda(), torch.from_numpy(pos).int().cuda(), torch.from_numpy(f).cuda())
    _check(out, x, pos, f, F32, far=True)
    # small angles keep their digits: y2 = x1 sin(p f) with p f from 1e-9 to 1e-3
    y, x1 = out[[1, 3], 1, 16 + 3].cpu().double().numpy(), x[[1, 3], 1, 3].double().numpy()
    want = x1 * np.sin(pos[[1, 3]] * 1e-9)
    assert np.all(np.abs(y - want) <= np.abs(want) * 2.0 ** -21)
    for bad in (float("inf"), float("nan"), 5e-324):  # count as 0
        out2 = torch.empty_like(out)
        pkv.rotary_embed(out2, x.cuda(), torch.from_numpy(pos).int().cuda(), torch.full((16,), bad, dtype=torch.float64).cuda())
        assert torch.equal(out2.cpu(), x)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,Hq,Hkv,D,R,off,B", [(1, 1, 1, 64, 64, 0, 8), (64, 32, 8, 128, 128, 0, 16), (37, 15, 3, 128, 48, 80, 32),
                                                (1001, 8, 8, 64, 32, 16, 16)])
def test_cache_write(dtype, T, Hq, Hkv, D, R, off, B):
    NB = -(-T // B) + 3
    qkv = _rows((T, Hq + 2 * Hkv, D), dtype, T)
    f = pkv.rotary_frequencies(R)
    r = np.random.default_rng(5)
    pos, slots = r.integers(0, 30000, T), r.permutation(NB * B)[:T]
    if T > 4:
        slots[2], slots[4] = -1, -(1 << 40)
    for inter in (False, True):
        dev = qkv.cuda()
        q, k, v = dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:]  # slices: strided tokens
        kc = torch.full((NB, Hkv, B, D), 7.0, dtype=dtype, device="cuda")
        vc = torch.full_like(kc, 7.0)
        sl, ps = torch.from_numpy(slots).cuda(), torch.from_numpy(pos).int().cuda()
        q_out = torch.empty(q.shape, dtype=dtype, device="cuda")
        assert pkv.kv_cache_write_rotary(k, v, kc, vc, sl, ps, f.cuda(), q=q, q_out=q_out, interleaved=inter, offset=off) is q_out
        assert torch.equal(dev.cpu(), qkv)
        assert pkv.read_device_errors(clear=True) == 0
        _check(q_out, qkv[:, :Hq], pos, f.numpy(), dtype, 1.0, inter, off)
        # the same bits as a rotation followed by the plain write; slots of no token left as they were
        rot = torch.empty((T, Hkv, D), dtype=dtype, device="cuda")
        pkv.rotary_embed(rot, k, ps, f.cuda(), interleaved=inter, offset=off)
        kc2, vc2 = torch.full_like(kc, 7.0), torch.full_like(vc, 7.0)
        pkv.kv_cache_write(rot, v.contiguous(), kc2, vc2, sl)
        assert torch.equal(kc, kc2) and torch.equal(vc, vc2)
        # in place, and without queries
        kc3, vc3 = torch.full_like(kc, 7.0), torch.full_like(vc, 7.0)
        pkv.kv_cache_write_rotary(k, v, kc3, vc3, sl, ps, f.cuda(), q=q, q_out=q, interleaved=inter, offset=off)
        assert torch.equal(q, q_out) and torch.equal(kc, kc3) and torch.equal(vc, vc3)
        kc3.fill_(7.0), vc3.fill_(7.0)
        pkv.kv_cache_write_rotary(k, v, kc3, vc3, sl, ps, f.cuda(), interleaved=inter, offset=off)
        assert torch.equal(kc, kc3) and torch.equal(vc, vc3)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,H,V,B", [(1, 1, 256, 8), (64, 32, 512, 16), (5, 0, 512, 64), (37, 5, 256, 32), (3001, 16, 512, 16)])
def test_latent_write(dtype, T, H, V, B):
    NB = -(-T // B) + 3
    rows = _rows((T, V + 64), dtype, T)
    qr = _rows((T, max(H, 1), 64), dtype, T + 1)
    f = pkv.rotary_frequencies(64, factor=8.0, original_len=4096.0)
    r = np.random.default_rng(6)
    pos, slots = r.integers(0, 100000, T), r.permutation(NB * B)[:T]
    if T > 4:
        slots[2], slots[4] = -1, -5
    dev = rows.cuda()
    cache = torch.full((NB, B, V + 64), 7.0, dtype=dtype, device="cuda")
    sl, ps = torch.from_numpy(slots).cuda(), torch.from_numpy(pos).int().cuda()
    q = torch.full((T, H, V + 64), 3.0, dtype=dtype, device="cuda")
    kw = dict(q_rope=qr.cuda(), q_out=q[..., V:]) if H else {}
    pkv.latent_cache_write(dev[:, :V], dev[:, V:], cache, sl, ps, f.cuda(), amplitude=1.2, interleaved=True, **kw)
    assert pkv.read_device_errors(clear=True) == 0
    ok = slots >= 0
    flat = cache.view(NB * B, V + 64).cpu()
    at = torch.from_numpy(slots[ok])
    assert torch.equal(flat[at][:, :V], rows[torch.from_numpy(ok)][:, :V])
    _check(flat[at][:, None, V:], rows[torch.from_numpy(ok)][:, None, V:], pos[ok], f.numpy(), dtype, 1.2, True)
    rest = np.setdiff1d(np.arange(NB * B), slots[ok])
    assert torch.all(flat[torch.from_numpy(rest)] == 7.0)
    if H:
        _check(q[..., V:], qr, pos, f.numpy(), dtype, 1.2, True)
        assert torch.all(q[..., :V] == 3.0)


def test_a_cache_past_32_bits():
    NB, Hkv, B, D, T = 140000, 8, 16, 128, 40  # 2.3e9 entries each
    kv = _rows((T, 2 * Hkv, D), BF, 5).cuda()
    ps, f = torch.arange(T, dtype=torch.int32, device="cuda"), pkv.rotary_frequencies(D, device="cuda")
    kc, vc = (torch.empty((NB, Hkv, B, D), dtype=BF, device="cuda") for _ in range(2))
    kc[-4:], vc[-4:] = 7.0, 7.0
    small = [torch.full((4, Hkv, B, D), 7.0, dtype=BF, device="cuda") for _ in range(2)]
    at = torch.randperm(4 * B, device="cuda")[:T]
    pkv.kv_cache_write_rotary(kv[:, :Hkv], kv[:, Hkv:], *small, at, ps, f)
    pkv.kv_cache_write_rotary(kv[:, :Hkv], kv[:, Hkv:], kc, vc, at + (NB - 4) * B, ps, f)
    assert torch.equal(kc[-4:], small[0]) and torch.equal(vc[-4:], small[1])


def test_bad_slots_are_flagged_and_skipped():
    T, Hkv, B, NB = 6, 2, 16, 2
    k = _rows((T, Hkv, 64), BF, 1).cuda()
    f, ps = pkv.rotary_frequencies(64, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
    slots = torch.tensor([0, NB * B, -1, 1 << 40, 2 ** 32, 31], device="cuda")
    kc = torch.full((NB, Hkv, B, 64), 7.0, dtype=BF, device="cuda")
    vc = torch.full_like(kc, 7.0)
    pkv.kv_cache_write_rotary(k, k, kc, vc, slots, ps, f)
    assert pkv.read_device_errors(clear=True) == pkv.DEVERR_SLOT
    want = torch.full_like(kc, 7.0)
    want[0, :, 0], want[1, :, 15] = k[0], k[5]  # positions 0: rows as they are
    assert torch.equal(kc, want) and torch.equal(vc, want)
    cache = torch.full((NB, B, 320), 7.0, dtype=BF, device="cuda")
    lat = _rows((T, 320), BF, 2).cuda()
    pkv.latent_cache_write(lat[:, :256], lat[:, 256:], cache, slots, ps, f)
    assert pkv.read_device_errors(clear=True) == pkv.DEVERR_SLOT
    want = torch.full_like(cache, 7.0)
    want[0, 0], want[1, 15] = lat[0], lat[5]
    assert torch.equal(cache, want)


def test_strided_heads_other_streams_and_graphs():
    T, H, D = 9, 4, 64
    base = _rows((H, T, D), BF, 1).cuda()
    x = base.transpose(0, 1)  # heads outermost
    ps = torch.arange(T, dtype=torch.int32, device="cuda") * 1000
    f = pkv.rotary_frequencies(64, device="cuda")
    want = torch.empty((T, H, D), dtype=BF, device="cuda")
    pkv.rotary_embed(want, x.contiguous(), ps, f)
    out = torch.empty_like(base).transpose(0, 1)
    pkv.rotary_embed(out, x, ps, f)
    assert torch.equal(out, want)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out2 = torch.empty_like(want)
    pkv.rotary_embed(out2, x, ps, f, stream=st)
    st.synchronize()
    assert torch.equal(out2, want)
    g = torch.cuda.CUDAGraph()
    out3 = torch.zeros_like(want)
    with torch.cuda.graph(g):
        pkv.rotary_embed(out3, x, ps, f)
    ps += 5
    pkv.rotary_embed(want, x, ps, f)
    g.replay()
    assert torch.equal(out3, want)


def test_refusals_on_the_device():
    x = torch.zeros((4, 2, 64), dtype=BF, device="cuda")
    ps, f = torch.zeros(4, dtype=torch.int32, device="cuda"), pkv.rotary_frequencies(64, device="cuda")
    with pytest.raises(TypeError):
        pkv.rotary_embed(x.half(), x.half(), ps, f)
    with pytest.raises(TypeError):
        pkv.rotary_embed(x.float(), x, ps, f)
    with pytest.raises(TypeError):
        pkv.rotary_embed(x, x, ps.long(), f)
    with pytest.raises(TypeError):
        pkv.rotary_embed(x, x, ps, f.float())
    with pytest.raises(TypeError):
        pkv.rotary_embed(x, x, ps, f.cpu())
    with pytest.raises(ValueError):
        pkv.rotary_embed(x, x, ps, f[None])
    with pytest.raises(ValueError):  # entries of a row apart
        pkv.rotary_embed(x, x.transpose(1, 2).contiguous().transpose(1, 2), ps, f)
    with pytest.raises(pkv.PkvError):  # rows not 16 bytes apart
        pkv.rotary_embed(x, torch.zeros((4, 2, 68), dtype=BF, device="cuda")[..., :64], ps, f)
    with pytest.raises(pkv.PkvError):  # every token written to one place
        pkv.rotary_embed(x[:1].expand(4, 2, 64), x, ps, f)
    with pytest.raises(ValueError):
        pkv.latent_cache_write(torch.zeros((4, 256), dtype=BF, device="cuda"), x[:, 0], torch.zeros((1, 16, 320), dtype=BF, device="cuda"),
                               torch.zeros(4, dtype=torch.int64, device="cuda"), ps, pkv.rotary_frequencies(32, device="cuda"))
    assert pkv.rotary_embed(x[:0], x[:0], ps[:0], f).shape[0] == 0
