"""The oracles of rotary positions and latent attention, pinned to invariants and to the other oracles."""
import numpy as np
import pytest
import torch

import paged_kv_cache_279_gb300 as pkv
from oracle import latent, rotary
from oracle.multi_token import multi_token_attention


def test_latent_attention_is_multi_token_attention_of_its_rows():
    r = np.random.default_rng(0)
    rows = r.standard_normal((23, 24))
    q = r.standard_normal((5, 3, 24))
    (out, spread, reach), = latent.latent_attention([q], [rows], 0.3, 16)
    v = np.concatenate([rows[:, :16], np.zeros((23, 8))], 1)
    ref, = multi_token_attention([q], [rows[:, None]], [v[:, None]], 0.3)
    np.testing.assert_allclose(out, ref[..., :16], rtol=0, atol=1e-12)
    assert np.all(spread >= np.abs(out) - 1e-12) and reach.shape == (5, 3, 1) and np.all(reach > 0)


def test_latent_attention_of_one_token_and_of_none():
    rows = np.random.default_rng(1).standard_normal((1, 24))
    q = np.random.default_rng(2).standard_normal((3, 2, 24))
    (out, _, _), = latent.latent_attention([q], [rows], 0.3, 16)
    assert np.all(out[:2] == 0.0)
    np.testing.assert_allclose(out[2], np.repeat(rows[:, :16], 2, 0), atol=1e-15)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_differences_of_positions(interleaved):
    r = np.random.default_rng(3)
    f = rotary.frequencies(16)
    q, k = r.standard_normal((1, 1, 24)), r.standard_normal((1, 1, 24))
    turned = lambda x, p: rotary.rotate(x, [p], f, 1.0, interleaved, 4)  # noqa: E731
    assert np.array_equal(turned(q, 0), q)
    assert np.linalg.norm(turned(q, 77)) == pytest.approx(np.linalg.norm(q))
    # the score depends on the difference of positions alone
    a = (turned(q, 1000) * turned(k, 990)).sum()
    assert a == pytest.approx((turned(q, 17) * turned(k, 7)).sum())
    assert np.array_equal(turned(q, 50)[..., :4], q[..., :4]) and np.array_equal(turned(q, 50)[..., 20:], q[..., 20:])
    # the two layouts are the same up to the order of entries
    if interleaved:
        order = np.concatenate([np.arange(4), 4 + 2 * np.arange(8), 5 + 2 * np.arange(8), np.arange(20, 24)])
        np.testing.assert_allclose(rotary.rotate(q[..., order], [9], f, 2.0, False, 4), rotary.rotate(q, [9], f, 2.0, True, 4)[..., order])


def test_far_angles():
    assert rotary.angle(0, 1.0) == 0.0
    assert rotary.angle(5, 1.0) == pytest.approx(5 - 2 * np.pi)
    assert np.cos(rotary.angle(10 ** 6, 0.1)) == pytest.approx(np.cos(10 ** 6 * 0.1), abs=1e-9)
    assert rotary.angle(-7, 0.3) == pytest.approx(-2.1)


@pytest.mark.parametrize("kw", [{}, {"base": 500000.0}, {"factor": 4.0}, {"factor": 8.0, "original_len": 4096.0},
                                {"factor": 32.0, "original_len": 8192.0, "low_turns": 1.0, "high_turns": 4.0}])
@pytest.mark.parametrize("R", [2, 64, 128])
def test_frequencies(R, kw):
    got = pkv.rotary_frequencies(R, **kw)
    assert got.dtype == torch.float64 and got.shape == (R // 2,)
    np.testing.assert_allclose(got.numpy(), rotary.frequencies(R, **kw), rtol=1e-14)
    assert got[0] <= 1.0 and torch.all(got[1:] < got[:-1])
