"""GPU: the row-scaled FP8 cache, bit-exact against its oracle, written and read back."""
import numpy as np
import pytest
import torch

import paged_kv_cache_279_gb300 as pkv
from oracle import fp8_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clear_errors():
    pkv.read_device_errors(clear=True)
    yield


def _rows(T, Hkv, D, dtype, seed):
    r = np.random.default_rng(seed)
    x = r.standard_normal((T, Hkv, D)) * np.exp(r.uniform(-30, 30, (T, Hkv, 1)))
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


def _pools(NB, Hkv, B, D, fill=0xA5):
    u8 = lambda *s: torch.full(s, fill, dtype=torch.uint8, device="cuda")  # noqa: E731
    return u8(NB, Hkv, B, D), u8(NB, Hkv, B, D), u8(NB, Hkv, B), u8(NB, Hkv, B)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,Hkv,D,B", [(1, 1, 64, 16), (1, 1, 128, 32), (7, 3, 64, 32), (33, 5, 128, 16), (200, 8, 128, 32)])
def test_write_is_exact_and_touches_only_its_slots(dtype, T, Hkv, D, B):
    NB = -(-T // B) + 3
    k, v = _rows(T, Hkv, D, dtype, 1), _rows(T, Hkv, D, dtype, 2)
    slots = np.random.default_rng(3).permutation(NB * B)[:T].astype(np.int64)
    if T > 4:
        slots[3] = -1
        slots[5] = -(1 << 40)
    kc, vc, ks, vs = _pools(NB, Hkv, B, D)
    pkv.kv_cache_write_fp8_rows(k.cuda(), v.cuda(), kc, vc, ks, vs, torch.from_numpy(slots).cuda())
    torch.cuda.synchronize()
    assert pkv.read_device_errors(clear=True) == 0
    for x, c, e in ((k, kc, ks), (v, vc, vs)):
        wc = np.full(c.shape, 0xA5, np.uint8)
        we = np.full(e.shape, 0xA5, np.uint8)
        codes, scales = fp8_rows.quantise_rows(x.float().numpy())
        ok = slots >= 0
        wc[slots[ok] // B, :, slots[ok] % B] = codes[ok]
        we[slots[ok] // B, :, slots[ok] % B] = scales[ok]
        assert np.array_equal(e.cpu().numpy(), we)
        assert np.array_equal(c.cpu().numpy(), wc)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("k_off,v_off", [(8, 8), (0, 8), (8, 0), (16, 16)])
def test_rows_on_any_16_byte_boundary(dtype, D, k_off, v_off):
    """Rows that begin 16 bytes (bf16) behind a 32-byte boundary give the same bytes, and are read back to such places."""
    T, Hkv, B = 37, 3, 16
    k, v = _rows(T, Hkv, D, dtype, 5).cuda(), _rows(T, Hkv, D, dtype, 6).cuda()

    def shifted(x, off):
        off = off if dtype == torch.bfloat16 else off // 2
        flat = torch.full((x.numel() + 32,), 7.0, dtype=dtype, device="cuda")
        y = flat[off:off + x.numel()].view(x.shape)
        y.copy_(x)
        return flat, y

    slots = torch.from_numpy(np.random.default_rng(3).permutation(5 * B)[:T].astype(np.int64)).cuda()
    want, got = _pools(5, Hkv, B, D), _pools(5, Hkv, B, D)
    pkv.kv_cache_write_fp8_rows(k, v, *want, slots)
    (_, ks), (_, vs) = shifted(k, k_off), shifted(v, v_off)
    pkv.kv_cache_write_fp8_rows(ks, vs, *got, slots)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    k2, v2 = torch.empty_like(k), torch.empty_like(v)
    pkv.kv_cache_read_fp8_rows(k2, v2, *want, slots)
    (kf, ks), (vf, vs) = shifted(torch.zeros_like(k), k_off), shifted(torch.zeros_like(v), v_off)
    pkv.kv_cache_read_fp8_rows(ks, vs, *want, slots)
    for plain, at, flat in ((k2, ks, kf), (v2, vs, vf)):
        assert torch.equal(plain, at)
        assert int((flat == 7.0).sum()) >= 32  # what lies around the rows is left


def test_write_of_special_rows():
    D, B = 64, 16
    x = torch.zeros(12, 1, D)
    x[0, 0, 5] = 448.0
    x[1, 0, 5] = 448.5
    x[2, 0, 63] = -450.0
    x[3, 0, 0] = 1e-45
    x[4, 0, :3] = torch.tensor([3.4e38, -3.4e38, 1.0])
    x[5, 0, :5] = torch.tensor([float("inf"), 1.0, float("-inf"), -2.0, 0.0])
    x[6, 0, :3] = torch.tensor([float("nan"), 5.0, -0.0])
    x[7, 0] = float("inf")
    x[8, 0, :4] = torch.tensor([1.0, 2.0 ** -17, 2.0 ** -18, 3 * 2.0 ** -18])
    x[9, 0] = -0.0
    x[10, 0, :2] = torch.tensor([2.0 ** -126, 2.0 ** -149])
    x[11, 0, :2] = torch.tensor([1.75, -1.0625])
    kc, vc, ks, vs = _pools(1, 1, B, D)
    pkv.kv_cache_write_fp8_rows(x.cuda(), x.cuda(), kc, vc, ks, vs, torch.arange(12).cuda())
    codes, scales = fp8_rows.quantise_rows(x.numpy())
    assert np.array_equal(ks[0, 0, :12].cpu().numpy(), scales[:, 0])
    got = kc[0, 0, :12].cpu().numpy()
    nan = (codes[:, 0] & 0x7F) == 0x7F
    assert np.array_equal(got[~nan], codes[:, 0][~nan]) and np.all((got[nan] & 0x7F) == 0x7F)
    assert torch.equal(kc, vc) and torch.equal(ks, vs)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,Hkv,D,B", [(1, 1, 64, 16), (7, 3, 64, 32), (33, 5, 128, 16), (300, 8, 128, 32)])
def test_read_returns_the_values(dtype, T, Hkv, D, B):
    NB = -(-T // B) + 2
    r = np.random.default_rng(4)
    pools = [r.integers(0, 256, (NB, Hkv, B, D)).astype(np.uint8) for _ in "kv"]
    scales = [r.integers(60, 200, (NB, Hkv, B)).astype(np.uint8) for _ in "kv"]
    slots = r.integers(0, NB * B, T).astype(np.int64)  # some twice
    if T > 2:
        slots[2] = -1
    out = [torch.full((T, Hkv, D), 9.0, dtype=dtype, device="cuda") for _ in "kv"]
    dev = [torch.from_numpy(x).cuda() for x in pools + scales]
    pkv.kv_cache_read_fp8_rows(*out, *dev, torch.from_numpy(slots).cuda())
    torch.cuda.synchronize()
    assert pkv.read_device_errors(clear=True) == 0
    for o, c, e in zip(out, pools, scales):
        want = fp8_rows.row_values(c[slots // B, :, slots % B], e[slots // B, :, slots % B])
        want[slots < 0] = 9.0
        assert np.array_equal(o.double().cpu().numpy(), want, equal_nan=True)  # every value is a bf16 number


def test_read_gives_back_what_was_written():
    T, Hkv, D, B = 500, 4, 128, 16
    k, v = _rows(T, Hkv, D, torch.bfloat16, 1).cuda(), _rows(T, Hkv, D, torch.bfloat16, 2).cuda()
    kc, vc, ks, vs = _pools(40, Hkv, B, D)
    slots = torch.randperm(40 * B)[:T].cuda()
    pkv.kv_cache_write_fp8_rows(k, v, kc, vc, ks, vs, slots)
    a, b = torch.empty_like(k), torch.empty_like(v)
    pkv.kv_cache_read_fp8_rows(a, b, kc, vc, ks, vs, slots)
    for x, y in ((k, a), (v, b)):
        amax = x.float().abs().amax(-1, keepdim=True)
        # half a step of 3 fraction bits, or of the subnormals (2^-10 of a scale that is at most amax / 224)
        assert torch.all((x.float() - y.float()).abs() <= torch.maximum(x.float().abs() * 2.0 ** -4, amax / 224 * 2.0 ** -10))
    kc2, vc2, ks2, vs2 = _pools(40, Hkv, B, D)
    pkv.kv_cache_write_fp8_rows(a, b, kc2, vc2, ks2, vs2, slots)  # its own values are fixed points up to the choice of scale
    c, d = torch.empty_like(k), torch.empty_like(v)
    pkv.kv_cache_read_fp8_rows(c, d, kc2, vc2, ks2, vs2, slots)
    assert torch.equal(a, c) and torch.equal(b, d)


def test_bad_slots_are_skipped_and_flagged():
    Hkv, D, B, NB = 2, 64, 16, 4
    k = torch.randn(3, Hkv, D, device="cuda")
    kc, vc, ks, vs = _pools(NB, Hkv, B, D)
    slots = torch.tensor([NB * B, 1 << 50, -3], device="cuda")
    pkv.kv_cache_write_fp8_rows(k, k, kc, vc, ks, vs, slots)
    assert pkv.read_device_errors(clear=True) == pkv.DEVERR_SLOT
    assert all(torch.all(x == 0xA5) for x in (kc, vc, ks, vs))
    out = torch.full((3, Hkv, D), 4.0, device="cuda")
    pkv.kv_cache_read_fp8_rows(out, out.clone(), kc, vc, ks, vs, slots)
    assert pkv.read_device_errors(clear=True) == pkv.DEVERR_SLOT
    assert torch.all(out == 4.0)


def test_blocks_and_scales_are_copied():
    Hkv, D, B, NB = 3, 64, 16, 6
    k = torch.randn(B, Hkv, D, device="cuda")
    kc, vc, ks, vs = _pools(NB, Hkv, B, D)
    pkv.kv_cache_write_fp8_rows(k, -k, kc, vc, ks, vs, torch.arange(2 * B, 3 * B, device="cuda"))
    pairs = torch.tensor([[2, 5]], device="cuda")
    pkv.block_copy([kc], [vc], pairs)
    pkv.block_copy([ks], [vs], pairs)
    torch.cuda.synchronize()
    for x in (kc, vc, ks, vs):
        assert torch.equal(x[5], x[2]) and torch.all(x[0] == 0xA5)


def test_captured_and_on_another_stream():
    Hkv, D, B, NB, T = 2, 128, 16, 8, 50
    k = torch.randn(T, Hkv, D, device="cuda", dtype=torch.bfloat16)
    slots = torch.randperm(NB * B)[:T].cuda()
    pools = _pools(NB, Hkv, B, D)
    out = torch.empty_like(k), torch.empty_like(k)

    def go():
        pkv.kv_cache_write_fp8_rows(k, k, *pools, slots)
        pkv.kv_cache_read_fp8_rows(*out, *pools, slots)
    go()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        go()
    torch.cuda.synchronize()
    for _ in range(3):
        k.mul_(1.5)
        g.replay()
        torch.cuda.synchronize()
        want = fp8_rows.row_values(*fp8_rows.quantise_rows(k.float().cpu().numpy()))
        assert np.array_equal(out[0].double().cpu().numpy(), want) and torch.equal(out[0], out[1])


def test_arguments_are_refused():
    Hkv, D, B, NB = 2, 128, 16, 4
    k = torch.randn(3, Hkv, D, device="cuda", dtype=torch.bfloat16)
    kc, vc, ks, vs = _pools(NB, Hkv, B, D)
    slots = torch.arange(3, device="cuda")
    f = pkv.kv_cache_write_fp8_rows
    with pytest.raises(TypeError):
        f(k.half(), k.half(), kc, vc, ks, vs, slots)
    with pytest.raises(TypeError):
        f(k, k.float(), kc, vc, ks, vs, slots)
    with pytest.raises(TypeError):
        f(k, k, kc, vc, ks, vs, slots.int())
    with pytest.raises(TypeError):
        f(k, k, kc, vc, ks.float(), vs, slots)
    with pytest.raises(ValueError):
        f(k, k, kc, vc, ks[:, :, :8], vs, slots)
    with pytest.raises(ValueError):
        f(k, k, kc, vc, ks, vs, slots[:2])
    with pytest.raises(ValueError):
        f(torch.randn(Hkv, 3, D, device="cuda", dtype=torch.bfloat16).transpose(0, 1), k, kc, vc, ks, vs, slots)
    with pytest.raises(TypeError):
        f(k.cpu(), k, kc, vc, ks, vs, slots)
    with pytest.raises(pkv.PkvError):  # blocks of 8
        f(k, k, *_pools(NB, Hkv, 8, D), slots)
    f(k[:0], k[:0], kc, vc, ks, vs, slots[:0])  # nothing to do
