"""The oracles of scored attention and of the row-scaled FP8 cache, pinned against independent statements (CPU only)."""
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import fp8_rows
from oracle.multi_token import multi_token_attention
from oracle.scored import scored_attention, seen_keys


def _draw(n, L, Hq, Hkv, D, seed):
    r = np.random.default_rng(seed)
    return r.standard_normal((n, Hq, D)), r.standard_normal((L, Hkv, D)), r.standard_normal((L, Hkv, D))


def test_without_options_it_is_the_plain_causal_attention():
    q, k, v = _draw(5, 23, 8, 2, 64, 1)
    out, _ = scored_attention(q, k, v, 0.125)
    assert np.abs(out - multi_token_attention([q], [k], [v], 0.125)[0]).max() < 1e-12
    out, _ = scored_attention(q[-1:], k, v, 0.125)
    assert np.abs(out - oracle.decode_attention(q[-1:], [k], [v], 0.125)).max() < 1e-6


@pytest.mark.parametrize("window,prefix,docs", [(0, 0, False), (4, 0, False), (1, 0, False), (6, 9, False), (0, 20, False),
                                                (5, 3, True), (0, 0, True)])
def test_masks_and_bias_against_torch_attention(window, prefix, docs):
    n, L, Hq, Hkv, D = 7, 19, 4, 2, 32
    q, k, v = _draw(n, L, Hq, Hkv, D, 2)
    starts = np.array([0, 0, 5, 5, 16, 16, 17]) if docs else None
    slopes = np.array([0.5, 0.25, 0.0, 1.0])
    out, _ = scored_attention(q, k, v, 0.2, slopes=slopes, window=window, prefix_len=prefix, key_starts=starts)
    bias = np.full((Hq, n, L), -np.inf)
    for h in range(Hq):  # the rule, key by key
        for i in range(n):
            p = L - n + i
            for t in range(L):
                ok = t < prefix or (t <= p and (window == 0 or p - t < window))
                if ok and (starts is None or t >= starts[i]):
                    bias[h, i, t] = -slopes[h] * abs(p - t)
    kk, vv = (torch.from_numpy(np.repeat(x, Hq // Hkv, axis=1)).permute(1, 0, 2) for x in (k, v))
    want = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q).permute(1, 0, 2), kk, vv,
                                                            attn_mask=torch.from_numpy(bias), scale=0.2)
    dead = np.isinf(bias).all(-1)
    want = np.where(dead[..., None], 0.0, np.nan_to_num(want.numpy()))
    assert np.abs(out - want.transpose(1, 0, 2)).max() < 1e-12


def test_cap_in_closed_form():
    # two keys with scores a and b: the weight of the first is the logistic of the capped difference
    q = np.zeros((1, 1, 2))
    q[0, 0] = [1.0, 0.0]
    k = np.array([[[300.0, 0.0]], [[7.0, 0.0]]])
    v = np.array([[[1.0, 0.0]], [[0.0, 1.0]]])
    out, _ = scored_attention(q, k, v, 0.1, softcap=5.0)
    x, y = 5 * math.tanh(30 / 5), 5 * math.tanh(0.7 / 5)
    assert abs(out[0, 0, 0] - 1 / (1 + math.exp(y - x))) < 1e-14
    # a cap far above every score changes nothing; a tiny one makes all weights equal
    q, k, v = _draw(3, 9, 2, 1, 16, 3)
    assert np.abs(scored_attention(q, k, v, 0.1, softcap=1e9)[0] - scored_attention(q, k, v, 0.1)[0]).max() < 1e-9
    assert np.abs(scored_attention(q[-1:], k, v, 0.1, softcap=1e-12)[0] - v.mean(0)).max() < 1e-9


def test_a_row_that_sees_nothing_is_zero():
    q, k, v = _draw(4, 6, 2, 2, 8, 4)
    out, _ = scored_attention(q, k, v, 1.0, key_starts=[0, 4, 6, 100])
    assert seen_keys([2, 3, 4, 5], 6, key_starts=[0, 4, 6, 100]).sum(1).tolist() == [3, 0, 0, 0]
    assert np.all(out[1:] == 0) and np.all(np.isfinite(out)) and np.any(out[0] != 0)


def test_row_exponent_and_codes():
    rows = np.zeros((9, 4))
    rows[0] = [448, -1, 0, 0]          # exactly the largest code
    rows[1] = [448.5, 0, 0, 0]         # just above: one binade up
    rows[2] = [0, 0, 0, 0]
    rows[3] = [2.0 ** -140, 0, 0, 0]   # below the smallest scale
    rows[4] = [3.3e38, -1e-30, 0, 0]
    rows[5] = [np.inf, 1.0, -2.0, np.nan]
    rows[6] = [1.75, 0, 0, 0]          # 448 * 2^-8
    rows[7] = [1.0, 2.0 ** -17, -2.0 ** -18, 0]
    rows[8] = [-1.7500001, 0, 0, 0]
    assert fp8_rows.row_exponent(rows).tolist() == [0, 1, -100, -100, 120, -7, -8, -8, -7]
    codes, scales = fp8_rows.quantise_rows(rows)
    vals = fp8_rows.row_values(codes, scales)
    assert scales.tolist() == [127, 128, 27, 27, 247, 120, 119, 119, 120]
    assert vals[0].tolist() == [448, -1, 0, 0] and vals[1][0] == 448 and vals[6][0] == 1.75
    assert vals[5][0] == 448 * 2.0 ** -7 and vals[5][1:3].tolist() == [1.0, -2.0] and np.isnan(vals[5][3])
    assert vals[7].tolist() == [1.0, 2.0 ** -17, -0.0, 0]  # half the smallest subnormal (2^-9 * 2^-8): to even
    assert codes[2].tolist() == [0, 0, 0, 0]


def test_row_values_lie_within_half_a_step_and_agree_with_torch():
    r = np.random.default_rng(5)
    x = (r.standard_normal((200, 64)) * np.exp(r.uniform(-20, 20, (200, 1)))).astype(np.float32)
    codes, scales = fp8_rows.quantise_rows(x)
    vals = fp8_rows.row_values(codes, scales)
    amax = np.abs(x).max(1, keepdims=True)
    # 3 fraction bits: half a step is 2^-4 of the value; subnormals: 2^-10 of the scale, at most amax / 224 (amax > 224 * 2^e)
    assert np.all(np.abs(vals - x) <= np.maximum(np.abs(x) * 2.0 ** -4, amax / 224 * 2.0 ** -10))
    y = torch.from_numpy(x.astype(np.float64) * np.exp2(127.0 - scales.astype(np.float64))[:, None])
    assert np.array_equal(y.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy(), codes)
