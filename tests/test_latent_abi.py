"""The rotary and latent attention calls refuse bad arguments on the host, before any device work (no GPU)."""
import ctypes

import pytest
import torch

import paged_kv_cache_279_gb300 as pkv
from paged_kv_cache_279_gb300 import _lib

P = ctypes.c_void_p(256)  # aligned, never dereferenced: each call below is refused before a launch
ODD = ctypes.c_void_p(264)
NAN, INF = float("nan"), float("inf")


def _str(*s):
    return (ctypes.c_int64 * len(s))(*s)


def _embed(p=None, x="p", T=4, H=8, D=128, R=128, off=0, st=None, amp=1.0, il=0, dt=1):
    return _lib.load().rotary_embed(p, p if x == "p" else x, p, p, T, H, D, R, off, st, amp, il, dt, None)


def _write(p=None, q="p", q_out="p", T=4, Hq=8, Hkv=2, D=128, R=128, off=0, B=16, NB=64, st=None, amp=1.0, il=0, dt=1):
    q, q_out = (p if x == "p" else x for x in (q, q_out))
    return _lib.load().kv_cache_write_rotary(q_out, q, p, p, p, p, p, p, p, T, Hq, Hkv, D, R, off, B, NB, st, amp, il, dt, None)


def _latent(p=None, q="p", q_out="p", T=4, H=8, V=512, B=16, NB=64, st=None, amp=1.0, il=0, dt=1):
    q, q_out = (p if x == "p" else x for x in (q, q_out))
    return _lib.load().latent_cache_write(q_out, q, p, p, p, p, p, p, T, H, V, B, NB, st, amp, il, dt, None)


@pytest.mark.parametrize("call", [_embed, _write, _latent])
def test_rotations(call):
    bad, no = pkv.PKV_ERR_INVALID, pkv.PKV_ERR_UNSUPPORTED
    assert call(ODD) == bad
    assert call(P, T=-1) == bad
    for a in (NAN, INF):
        assert call(P, amp=a) == bad
    assert call(P, il=2) == bad
    assert call(P, dt=2) == no
    assert call(None, T=4) == bad
    ok = dict(Hq=0) if call is _write else dict(H=0) if call is _latent else {}
    assert call(None, T=0, **ok) == pkv.PKV_OK
    n = {_embed: 4, _write: 8, _latent: 6}[call]
    fine = [1024, 128] * (n // 2)
    for i in range(n):  # no multiple of 16 bytes; too far
        for x in (1028, 1 << 60):
            assert call(P, st=_str(*fine[:i], x, *fine[i + 1:])) == bad
    assert call(P, st=_str(0, *fine[1:])) == bad         # two tokens written to one place
    assert call(P, st=_str(1024, 0, *fine[2:])) == bad   # two heads


@pytest.mark.parametrize("call", [_embed, _write])
def test_rotated_part(call):
    bad, no = pkv.PKV_ERR_INVALID, pkv.PKV_ERR_UNSUPPORTED
    assert call(P, R=0) == bad and call(P, R=144) == bad and call(P, R=64, off=80) == bad and call(P, off=-16, R=64) == bad
    assert call(P, R=64, off=2 ** 31 - 16) == bad
    assert call(P, R=24) == no and call(P, R=64, off=8) == no and call(P, D=100, R=16) == no
    assert call(P, D=0, R=16) == bad


def test_their_own():
    bad, no = pkv.PKV_ERR_INVALID, pkv.PKV_ERR_UNSUPPORTED
    assert _embed(P, H=0) == bad and _embed(P, D=512, R=512) == no and _embed(P, H=2 ** 31 - 1) == no
    assert _embed(P, x=None) == bad
    assert _write(P, D=96, R=96) == no and _write(P, B=64) == no and _write(P, B=12) == no
    assert _write(P, Hkv=0) == bad and _write(P, NB=0) == bad and _write(P, Hq=-1) == bad
    assert _write(P, q=None) == bad and _write(P, q_out=None) == bad and _write(P, Hq=0) == bad
    assert _write(P, Hkv=2 ** 31 - 1) == no
    assert _latent(P, V=384) == no and _latent(P, V=0) == bad and _latent(P, B=24) == no and _latent(P, NB=0) == bad
    assert _latent(P, q=None) == bad and _latent(P, q_out=None) == bad and _latent(P, H=0) == bad
    assert _latent(P, H=2 ** 31 - 1) == no


def test_frequencies():
    f = _lib.load().rotary_frequencies
    out = (ctypes.c_double * 4)()
    bad = pkv.PKV_ERR_INVALID
    assert f(out, 8, 1e4, 1.0, 0.0, 1.0, 32.0) == pkv.PKV_OK and out[0] == 1.0
    assert f(None, 8, 1e4, 1.0, 0.0, 1.0, 32.0) == bad and f(out, 7, 1e4, 1.0, 0.0, 1.0, 32.0) == bad
    assert f(out, 0, 1e4, 1.0, 0.0, 1.0, 32.0) == bad
    for x in (0.0, -1.0, NAN, INF):
        assert f(out, 8, x, 1.0, 0.0, 1.0, 32.0) == bad and f(out, 8, 1e4, x, 0.0, 1.0, 32.0) == bad
    for x in (-1.0, NAN, INF):
        assert f(out, 8, 1e4, 2.0, x, 1.0, 32.0) == bad
    assert f(out, 8, 1e4, 2.0, 4096.0, 32.0, 1.0) == bad and f(out, 8, 1e4, 2.0, 4096.0, 1.0, NAN) == bad
    with pytest.raises(ValueError):
        pkv.rotary_frequencies(7)
    with pytest.raises(pkv.PkvError):
        pkv.rotary_frequencies(8, base=-1.0)


def _decode(p=None, S=2, H=16, V=512, B=16, maxB=4, NB=16, maxL=64, scale=0.1, ws=P, nws=1 << 40, dt=1):
    return _lib.load().paged_latent_attention_decode(p, p, p, p, p, S, H, V, B, maxB, NB, maxL, scale, ws, nws, dt, None)


def _multi(p=None, S=2, T=10, H=16, V=512, B=16, maxB=4, NB=16, maxQ=5, maxL=64, scale=0.1, ws=P, nws=1 << 40, dt=1):
    return _lib.load().paged_latent_attention_multi_token(p, p, p, p, p, p, S, T, H, V, B, maxB, NB, maxQ, maxL, scale, ws,
                                                          nws, dt, None)


@pytest.mark.parametrize("call", [_decode, _multi])
def test_attention_calls(call):
    bad, no = pkv.PKV_ERR_INVALID, pkv.PKV_ERR_UNSUPPORTED
    assert call() == bad                                       # null pointers
    assert call(ODD) == bad
    assert call(P, S=-1) == bad and call(P, H=0) == bad and call(P, maxB=0) == bad and call(P, NB=0) == bad
    assert call(P, maxL=-1) == bad and call(P, B=0) == bad and call(P, V=0) == bad
    assert call(P, H=129) == no and call(P, V=384) == no and call(P, V=1024) == no and call(P, B=12) == no
    assert call(P, dt=2) == no
    for x in (NAN, INF, 3e38, -3e38):
        assert call(P, scale=x) == bad
    assert call(P, maxB=1 << 28) == bad                        # positions past 31 bits
    assert call(P, NB=1 << 28) == no                           # cache rows past 31 bits
    assert call(P, ws=None) == bad and call(P, ws=ODD) == bad and call(P, nws=16) == bad
    assert call(S=0) == pkv.PKV_OK


def test_multi_token_only():
    assert _multi(P, maxQ=0) == pkv.PKV_ERR_INVALID and _multi(P, T=-1) == pkv.PKV_ERR_INVALID
    assert _multi(P, T=2 ** 31 - 1) == pkv.PKV_ERR_UNSUPPORTED
    assert _multi(T=0) == pkv.PKV_OK


def test_workspace_sizes():
    f = _lib.load().paged_latent_attention_workspace_size
    for dt in (0, 1):
        assert f(0, 16, 512, 100, dt) == 0 and f(4, 0, 512, 100, dt) == 0 and f(4, 16, 100, 100, dt) == 0
        assert f(4, 16, 512, 0, dt) == 0
        assert f(4, 16, 512, 10000, dt) > 0 and f(4, 16, 512, 10000, dt) % 256 == 0
        # no call with a smaller table or a shorter context needs more
        assert f(4, 16, 512, 100, dt) <= f(4, 16, 512, 10000, dt)
    assert f(4, 16, 512, 100, 2) == 0
    with pytest.raises(TypeError):
        pkv.paged_latent_attention_workspace_size(4, 16, 512, 100, torch.float16)


def test_python_refusals():
    x = torch.zeros(4, 8, 128)
    pos, f = torch.zeros(4, dtype=torch.int32), pkv.rotary_frequencies(128)
    with pytest.raises(TypeError):                             # not on a GPU
        pkv.rotary_embed(x, x, pos, f)
    with pytest.raises(ValueError):
        pkv.rotary_embed(x[:2], x, pos, f)
    with pytest.raises(ValueError):
        pkv.rotary_embed(x, x, pos[:3], f)
    kc = torch.zeros(2, 8, 16, 128)
    slots = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        pkv.kv_cache_write_rotary(x, x, kc, kc, slots, pos, f, q=x)
    with pytest.raises(ValueError):
        pkv.kv_cache_write_rotary(x, x[:3], kc, kc, slots, pos, f)
    with pytest.raises(ValueError):
        pkv.kv_cache_write_rotary(x, x, kc, kc, slots[:3], pos, f)
    with pytest.raises(TypeError):
        pkv.kv_cache_write_rotary(x, x, kc, kc, slots, pos, f)
    cache = torch.zeros(2, 16, 576)
    with pytest.raises(ValueError):
        pkv.latent_cache_write(torch.zeros(4, 256), x[:, 0, :64], cache, slots, pos, f)
    with pytest.raises(TypeError):
        pkv.latent_cache_write(torch.zeros(4, 512), x[:, 0, :64], cache, slots, pos, f[:32])
    with pytest.raises(ValueError):
        pkv.latent_cache_write(torch.zeros(4, 512), x[:, 0, :64], cache, slots, pos, f)
    q, out = torch.zeros(2, 16, 576), torch.zeros(2, 16, 512)
    tables, lens = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        pkv.paged_latent_attention_decode(out, q[..., :320], cache, tables, lens, 0.1, 16)
    with pytest.raises(ValueError):
        pkv.paged_latent_attention_decode(out[:1], q[:1], cache, tables, lens, 0.1, 16)
    with pytest.raises(TypeError):
        pkv.paged_latent_attention_decode(out, q, cache, tables, lens, 0.1, 16)
    with pytest.raises(ValueError):
        pkv.paged_latent_attention_multi_token(out, q, cache, tables, lens, lens, 0.1, 1, 16)
