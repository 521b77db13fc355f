"""Scored attention at the ends of its ranges: V rows of very different sizes, wide caps, extreme scales."""
import copy

import numpy as np
import pytest
import torch

import paged_kv_cache_279_gb300 as pkv
from oracle import fp8_rows
from scored_cases import Case
from test_gpu_scored import run

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_errors():
    pkv.read_device_errors(clear=True)
    yield
    assert pkv.read_device_errors(clear=True) == 0


def _rows_case(n, scores, sizes):
    """One row-scaled FP8 context of n tokens: q.k is scores[t], V rows are normal times sizes[t]."""
    c = Case([n], 2, 1, 64, 16, rows=True, scale=1.0)
    c.q[:] = 0
    c.q[..., 0] = 1.0
    k = np.zeros((n, 1, 64), np.float32)
    k[:, 0, 0] = scores
    v = (np.random.default_rng(8).standard_normal((n, 1, 64)) * np.asarray(sizes, np.float64)[:, None, None]).astype(np.float32)
    c.codes = [(fp8_rows.quantise_rows(k), fp8_rows.quantise_rows(v))]
    c.ks, c.vs = ([torch.from_numpy(fp8_rows.row_values(*p))] for p in c.codes[0])
    return c


@pytest.mark.parametrize("apart", [0.0, -20.75, 20.75])
@pytest.mark.parametrize("small", [0.0, 2.0 ** -97], ids=["zero", "tiny"])
def test_rows_long_runs_of_small_values(small, apart):
    """Half of a long context has V rows of zeros (or of about 2^-97), whose scale is the least there is: the sum of the
    weights stays finite whatever the order of the halves."""
    n = 40000
    first = np.arange(n) < n // 2
    for head in (first, ~first):
        c = _rows_case(n, np.where(head, apart, 0.0), np.where(head, small, 1.0))
        c.check(run(c))


@pytest.mark.parametrize("large", [2.0 ** 30, 2.0 ** 60, 2.0 ** 110])
@pytest.mark.parametrize("n", [60, 300, 5000])
def test_rows_zeros_beside_large_values(n, large):
    """Zero rows keep their part of the sum when rows up to 2^200 times the least scale follow or precede them."""
    first = np.arange(n) < n // 2
    for head in (first, ~first):
        c = _rows_case(n, np.zeros(n), np.where(head, 0.0, large))
        c.check(run(c))
    # everything tiny: a row of any size keeps its precision
    c = _rows_case(n, np.linspace(0, 3, n), np.full(n, 2.0 ** -97))
    c.check(run(c))


@pytest.mark.parametrize("cap,hot", [(60.0, 15.0), (1e4, 1500.0), (1e6, 1.5e5), (1e9, 1.5e8)])
@pytest.mark.parametrize("kind", ["rows", "bf16", "multi", "alibi"])
def test_a_wide_cap_that_others_reach(kind, cap, hot):
    """One head's scores reach a wide cap: the other heads' results, far below it, are as good as without it (the bound is
    the uncapped one, plus 2^-19 of a score)."""
    c = Case([77, 300], qlens=[9, 130] if kind in ("multi", "alibi") else None, rows=kind == "rows", softcap=cap, window=90,
             alibi=kind == "alibi")
    ref, _ = c.reference()
    plain = copy.copy(c)
    plain.softcap = 0.0
    _, tol = plain.reference()
    rep, at = c.Hq // c.Hkv, 0
    for s, L in enumerate(c.lens):
        n = int(c.q_starts[s + 1] - c.q_starts[s])
        q, k = (x.double().abs().numpy() for x in (c.q[at:at + n], c.ks[s]))
        a = c.scale * max(float((q[:, h] @ k[:, h // rep].T).max()) for h in range(c.Hq))
        tol[at:at + n] += 4 * 2.0 ** -19 * a * c.vs[s].double().abs().max().item()
        at += n
    c.q = c.q.clone()
    c.q[:, 1] *= hot
    got = run(c).double().cpu().numpy()
    others = [h for h in range(c.Hq) if h != 1]
    assert np.all(np.abs(got - ref)[:, others] <= tol[:, others])


@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e-7, 1e-4, 1e4, 1e7, 1e12, 1e30])
@pytest.mark.parametrize("cap", [12.0, 200.0])
@pytest.mark.parametrize("kind", ["f32", "bf16", "rows", "multi"])
def test_extreme_scales(kind, cap, scale):
    """Scores of ordinary size made of very large queries and a tiny scale, or the other way round."""
    c = Case([77, 300], qlens=[9, 130] if kind == "multi" else None, rows=kind == "rows", softcap=cap, scale=scale,
             qmul=2.0 / scale / 128 ** 0.5, dtype=torch.float32 if kind == "f32" else torch.bfloat16)
    c.check(run(c))


@pytest.mark.parametrize("scale", [0.0, -0.1, 0.3])
@pytest.mark.parametrize("kind", ["f32", "bf16", "rows", "multi"])
def test_plain_scores_of_any_scale(kind, scale):
    """No cap and no bias, scores of either sign."""
    c = Case([77, 300, 900], qlens=[9, 130, 33] if kind == "multi" else None, rows=kind == "rows", scale=scale, window=250,
             dtype=torch.float32 if kind == "f32" else torch.bfloat16)
    c.check(run(c))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sign,size", [(1.0, 2.0 ** 50), (-1.0, 2.0 ** 50), (1.0, 2.0 ** -30), (-1.0, 2.0 ** -30), (1.0, 2.0 ** 112),
                                       (-1.0, 2.0 ** 112)])
def test_multi_values_at_the_ends_of_a_cap(sign, size, D):
    """Every score at +-50, V large or small: what the fixed reference of capped scores holds, and where it would overflow."""
    c = Case([900, 40], 4, 1, D, 16, qlens=[140, 40], softcap=50.0, scale=1.0)
    c.q = c.q.abs() + 8.0
    c.ks = [(sign * (k.abs() + 8.0)) for k in c.ks]
    c.vs = [v * size for v in c.vs]
    c.check(run(c))


@pytest.mark.parametrize("cap", [0.0, 5.0])
@pytest.mark.parametrize("kind", ["f32", "bf16", "multi"])
def test_scores_of_minus_infinity(kind, cap):
    """Keys whose scores are -infinity, whole runs of them at either end: weights of zero, or a cap's lower end."""
    n = 700
    c = Case([n, 40], 4, 1, 64, 16, qlens=[60, 5] if kind == "multi" else None, softcap=cap, scale=0.1,
             dtype=torch.float32 if kind == "f32" else torch.bfloat16)
    c.q[..., 3] = 1.0
    low = [np.r_[0:300, 420:430, 600:n - 60], np.r_[0:20]]
    for k, t in zip(c.ks, low):
        k[t, :, 3] = -float("inf")
    pools = c.pools()
    for k, t in zip(c.ks, low):
        k[t, :, 3] = -1e30   # the same to 64 bits: exp(-1e29) is 0, tanh(-2e28) is -1
    ref, _ = c.reference()
    # the bound of scored_cases with sizes of ordinary scores (scale sum |q||k| below 64) and vmax for sum_t w_t |v_t|
    vmax = max(v.double().abs().max().item() for v in c.vs)
    x = (64 + 16) * 2.0 ** -24 * 64 + 2.0 ** -20 + 2.0 ** -18 * cap + 2.0 ** -22 * 64
    weight = 0.0 if kind == "f32" else 2.0 ** -8
    tol = 2 * (2 * x + weight + n * 2.0 ** -24) * vmax + torch.finfo(c.dtype).eps / 2 * np.abs(ref) * (1 + 2.0 ** -6)
    got = run(c, pools).double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= tol)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("opt", [{}, dict(alibi=True), dict(softcap=50.0), dict(softcap=50.0, alibi=True), dict(softcap=200.0)],
                         ids=["plain", "alibi", "cap", "cap_alibi", "wide_cap"])
@pytest.mark.parametrize("kind", ["f32", "bf16", "multi"])
def test_very_large_values(kind, opt, D):
    """V of 2^112 under scores that rise along the context by 40: weights relative to the first keys would overflow."""
    c = Case([900, 300], 4, 1, D, 16, qlens=[140, 33] if kind == "multi" else None,
             dtype=torch.float32 if kind == "f32" else torch.bfloat16, scale=1.0, **opt)
    c.q = (0.05 * c.q.float()).to(c.dtype)
    c.q[..., 0] = 1.0
    for s, L in enumerate(c.lens):
        c.ks[s][:, 0, 0] = torch.linspace(-20.0, 20.0, L).to(c.dtype)
    c.vs = [v * 2.0 ** 112 for v in c.vs]
    c.check(run(c))
