"""GPU: latent attention where scores pass float32's range, or scores or latent entries are very large."""
import numpy as np
import pytest
import torch

import latent_cases as lc
import latent_more as lm
import paged_kv_cache_279_gb300 as pkv

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _clear_errors():
    pkv.read_device_errors(clear=True)
    yield
    assert pkv.read_device_errors(clear=True) == 0


def _tokens(which, L):
    t = np.zeros(L, dtype=bool)
    if which == "last":
        t[-1] = True
    elif which == "early":
        t[5] = True
    elif which == "several":
        t[np.random.default_rng(L).permutation(L)[:L // 3]] = True
    elif which == "tail":
        t[L - L % 48 - 1:] = True
    elif which == "all":
        t[:] = True
    return t


def _overflow(which, heads, H, V, dtype, queries, at, sign=-1.0, lens=(150, 77), power=64, B=16):
    """A case of finite numbers, some products 2^(2 power + 1) in size: (case, dead tokens a sequence)."""
    c = lc.make(list(lens), H, V, B, dtype, queries, seed=3, fill=0.0)
    e = V + 5 if at == "key" else 9
    some = np.ones(H, dtype=bool) if heads == "all" else np.arange(H) % 2 == 1
    c["q"][:, :, e] = torch.from_numpy(np.where(some, 2.0 ** power, 0.0)).to(dtype)
    dead = []
    for x in c["rows"]:
        t = _tokens(which, x.shape[0])
        x[:, e] = torch.from_numpy(np.where(t, sign * 2.0 ** (power + 1), 0.0)).to(dtype)
        dead.append(some[:, None] & t[None])
    return lm.store(c), dead


# up to 64 rows of a sequence
FEW = [(1, None, 512, BF), (16, None, 512, BF), (33, None, 256, BF), (64, None, 512, BF), (1, [3, 2], 512, BF), (4, [9, 5], 512, BF),
       (16, [4, 2], 256, BF)]
MANY = [(128, None, 512, BF), (100, None, 256, BF), (16, [40, 9], 512, BF), (6, [70, 30], 256, BF), (1, [140, 70], 512, BF)]


def _hidden_by_overflow(which, heads, H, queries, V, dtype, at, sign, table, power=64):
    c, dead = _overflow(which, heads, H, V, dtype, queries, at, sign, power=power)
    if table:
        c = lm.wide(c, table)
    scale = lc.SCALE if sign < 0 else -lc.SCALE
    got = lc.run(c, scale=scale, max_len=10 ** 6)
    lm.check(got, lm.expected(c, dead, scale))
    if which == "all":  # every score of these heads is -infinity
        assert torch.all(got[:, dead[0][:, 0]] == 0)


WHERE = [("last", "all", "key", -1.0), ("early", "all", "key", -1.0), ("several", "some", "key", -1.0),
         ("several", "all", "latent", -1.0), ("tail", "some", "latent", 1.0),
         ("tail", "all", "key", -1.0), ("all", "all", "key", 1.0), ("all", "some", "key", -1.0)]


@pytest.mark.parametrize("table", [0, 8192])
@pytest.mark.parametrize("which,heads,at,sign", WHERE)
@pytest.mark.parametrize("H,queries,V,dtype", FEW)
def test_scores_below_all_numbers(H, queries, V, dtype, which, heads, at, sign, table):
    """Products of finite entries that pass 3.4e38: scores of -infinity, weights of 0, wherever the tokens lie."""
    _hidden_by_overflow(which, heads, H, queries, V, dtype, at, sign, table)


@pytest.mark.parametrize("table", [0, 8192])
@pytest.mark.parametrize("which,heads,at,sign", WHERE)
@pytest.mark.parametrize("H,queries,V,dtype", MANY)
def test_scores_below_all_numbers_on_pairs(H, queries, V, dtype, which, heads, at, sign, table):
    """The same for more than 64 query rows a sequence."""
    _hidden_by_overflow(which, heads, H, queries, V, dtype, at, sign, table)


@pytest.mark.parametrize("which,heads,at,sign", WHERE)
@pytest.mark.parametrize("H,queries,V", [(5, None, 512), (3, [9, 5], 256)])
def test_float32_scores_below_all_numbers(H, queries, V, which, heads, at, sign):
    """The same in float32, which scales queries before the products: 2^133 times 0.104 (scale and log2 e) passes its range,
    2^129 times that does not."""
    _hidden_by_overflow(which, heads, H, queries, V, F32, at, sign, 0, power=66)


@pytest.mark.parametrize("dtype,H,queries", [(BF, 16, None), (F32, 5, None), (BF, 4, [9, 5])])
def test_an_infinite_query_whose_scores_are_all_minus_infinity(dtype, H, queries):
    c = lc.make([150, 77], H, 512, 16, dtype, queries, fill=0.0)
    for x in c["rows"]:
        x[:, 520] = -1.0
    want = lc.run(lm.store(c))
    c["q"][:, 2, 520] = float("inf")
    got = lc.run(c)
    assert torch.all(got[:, 2] == 0)
    keep = torch.arange(H) != 2
    assert torch.equal(got[:, keep], want[:, keep])


def _bad_row_beside(H, queries, at, bad, table, V=512, B=16):
    """Token 60 holds something that is no number, 57 and 70 have scores of -infinity: who does not see 60 is not touched by it."""
    c, dead = _overflow("none", "all", H, V, BF, queries, "key", lens=(90, 77), B=B)
    e = V + 5
    for t in (57, 70):
        c["rows"][0][t, e] = -2.0 ** 65
        dead[0][:, t] = True
    c = lm.store(lm.wide(c, table) if table else c)
    want = lc.run(c, max_len=10 ** 6)
    lm.check(want, lm.expected(c, dead))
    cache = c["cache"].clone()
    cache[int(c["tables"][0][60 // B]), 60 % B, at] = bad
    got = lc.run(c, cache=cache.cuda(), max_len=10 ** 6)
    n = c["nq"][0]
    sees = torch.zeros(want.shape[0], dtype=torch.bool)
    sees[max(0, 60 - (90 - n)):n] = True
    assert torch.equal(got[~sees.cuda()], want[~sees.cuda()])
    if at < V or bad != bad:
        assert torch.all(~torch.isfinite(got[sees.cuda()][..., min(at, V - 1)]))


@pytest.mark.parametrize("at", [33, 512 + 40])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("table", [0, 8192])
@pytest.mark.parametrize("H,queries", [(1, [40, 9]), (2, [32, 3]), (16, [4, 4]), (16, None)])
def test_a_row_that_is_no_number_beside_such_scores(H, queries, at, bad, table):
    _bad_row_beside(H, queries, at, bad, table)


@pytest.mark.parametrize("at", [33, 300, 512 + 40])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("table", [0, 8192])
@pytest.mark.parametrize("H,queries", [(2, [50, 9]), (16, [40, 9]), (128, None), (70, [3, 2])])
def test_a_row_that_is_no_number_beside_such_scores_on_pairs(H, queries, at, bad, table):
    _bad_row_beside(H, queries, at, bad, table)


@pytest.mark.parametrize("at", [0, 130, 255])
@pytest.mark.parametrize("bad", [float("nan"), -float("inf")])
@pytest.mark.parametrize("table", [0, 8192])
@pytest.mark.parametrize("H,queries,B", [(64, None, 8), (2, [25, 9], 64), (5, [3, 2], 32), (2, [50, 9], 8), (100, None, 64)])
def test_a_row_that_is_no_number_in_256_entries(H, queries, B, at, bad, table):
    _bad_row_beside(H, queries, at, bad, table, V=256, B=B)


def test_an_infinite_query_on_pairs_whose_scores_are_all_minus_infinity():
    for H, queries in ((100, None), (5, [30, 20])):
        c = lc.make([150, 77], H, 512, 16, BF, queries, fill=0.0)
        for x in c["rows"]:
            x[:, 520] = -1.0
        want = lc.run(lm.store(c))
        c["q"][:, 2, 520] = float("inf")
        got = lc.run(c)
        assert torch.all(got[:, 2] == 0)
        keep = torch.arange(H) != 2
        assert torch.equal(got[:, keep], want[:, keep])


def _sparse(H, V, dtype, queries, top, order, seed=7, lens=(150, 600)):
    """Integers times a power of two, 24 entries of a query not zero: products and their sums are exact in float32 (up to the
    scale), scores up to about ``top``."""
    c = lc.make(list(lens), H, V, 16, dtype, queries, seed=seed, fill=0.0)
    r = np.random.default_rng(seed)
    T = c["q"].shape[0]
    q = np.zeros((T, H, V + 64))
    for t in range(T):
        for h in range(H):
            q[t, h, r.permutation(V + 64)[:24]] = r.integers(1, 9, 24) * r.choice([-1, 1], 24)
    c["q"] = torch.from_numpy(q).to(dtype)
    for x in c["rows"]:
        y = r.integers(-8, 9, tuple(x.shape)).astype(np.float64)
        if order:  # scores that rise or fall along the context
            y *= 2.0 ** np.round(np.linspace(-3, 3, x.shape[0]) * order)[:, None]
        x.copy_(torch.from_numpy(y).to(dtype))
    biggest = max(np.abs(c["q"].double().numpy() @ x.double().numpy().T).max() for x in c["rows"])
    return lm.store(c), top / biggest


def _large_scores(H, V, dtype, queries, top, order, table):
    c, scale = _sparse(H, V, dtype, queries, top, order)
    scale = float(np.float32(scale))
    if table:
        c = lm.wide(c, table)
    for sc in (scale, -scale):
        want, tol = lm.expected(c, lm.none_dead(c), sc, terms=24, moves=2 + 600 // 48)
        live = np.abs(want) > 1e-30
        assert np.mean(np.abs(want[live]) > 4 * tol[live]) > 0.9  # (zeros, or signs turned, would not do)
        lm.check(lc.run(c, scale=sc, max_len=10 ** 6), (want, tol))


@pytest.mark.parametrize("table", [0, 8192])
@pytest.mark.parametrize("top,order", [(30.0, 0), (1000.0, 0), (1000.0, 1), (1000.0, -1)])
@pytest.mark.parametrize("H,V,dtype,queries", [(9, 512, BF, None), (64, 256, BF, None), (128, 512, BF, None), (4, 512, BF, [9, 3]), (5, 256, BF, [40, 3]),
                                               (5, 512, F32, None), (3, 256, F32, [9, 3])])
def test_large_scores(H, V, dtype, queries, top, order, table):
    _large_scores(H, V, dtype, queries, top, order, table)


@pytest.mark.parametrize("rise", [0.0, 5.4, 100.0])
@pytest.mark.parametrize("H,dtype,queries", [(9, BF, None), (64, BF, None), (100, BF, None), (5, BF, [40, 3]), (5, F32, None)])
def test_the_largest_latent_entries(H, dtype, queries, rise):
    """Just below 2^120 over the tokens in bf16, 2^128 over them in float32: the sums stay finite, also where scores rise along
    the context, by almost 2^8 in weight before the reference moves, or by far more."""
    c = lc.make([255, 100], H, 512, 16, dtype, queries, fill=0.0)
    c["q"][..., :512] = 0.0  # (the latent entries are part of the keys)
    c["q"][..., 512:] *= 0.1
    c["q"][..., 575] = 1.0
    for x in c["rows"]:
        x[:, :512] = (torch.sign(x[:, :512].float()) * (2.0 ** 112 if dtype == BF else 2.0 ** 120)).to(dtype)
        x[:, :7] = x[:, :7].abs()  # entries whose sums do not cancel
        x[:, 575] = torch.linspace(0.0, rise / lc.SCALE, x.shape[0]).to(dtype)
    lc.check(lc.run(lm.store(c)), c)
    lc.check(lc.run(lm.wide(c), max_len=10 ** 6), c)
