"""Several queries a sequence: what stands in keys that a query does not see has no effect on it, also where other
queries of the same sequence see them."""
import numpy as np
import pytest
import torch

import paged_kv_cache_279_gb300 as pkv
from harness import bits
from oracle.scored import seen_keys
from scored_cases import Case
from test_gpu_scored import run

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_errors():
    pkv.read_device_errors(clear=True)
    yield
    assert pkv.read_device_errors(clear=True) == 0


def check_poisoned(c: Case, bad):
    """bad: (sequence, key, kv head or slice, column or slice, value).  Outputs that see none of them are right, the others
    are not finite."""
    pools = c.pools()
    hit = [np.zeros((L, c.Hkv, c.D), bool) for L in c.lens]
    for s, t, g, col, x in bad:
        pools["v_cache"][int(c.tables[s][t // c.B]), g, t % c.B, col] = x
        hit[s][t, g, col] = True
    saved = c.vs
    c.vs = [torch.where(torch.from_numpy(h), torch.zeros_like(v), v) for h, v in zip(hit, c.vs)]
    ref, tol = c.reference()
    c.vs = saved
    spoilt = np.zeros(ref.shape, bool)
    for s, L in enumerate(c.lens):
        a, b = int(c.q_starts[s]), int(c.q_starts[s + 1])
        seen = seen_keys(np.arange(L - (b - a), L), L, c.window, 0 if c.prefix is None else min(max(0, c.prefix[s]), L),
                         None if c.starts is None else c.starts[a:b])
        for g in range(c.Hkv):
            n = c.Hq // c.Hkv
            spoilt[a:b, g * n:(g + 1) * n] = (seen.astype(np.float64) @ hit[s][:, g].astype(np.float64) > 0)[:, None]
    got = run(c, pools)
    assert torch.equal(bits(got), bits(run(c, pools)))
    x = got.double().cpu().numpy()
    assert spoilt.any() or not bad
    assert not np.isfinite(x[spoilt]).any()
    assert np.isfinite(x[~spoilt]).all(), f"{(~np.isfinite(x[~spoilt])).sum()} of {(~spoilt).sum()} outputs spoilt by keys they do not see"
    assert (np.abs(x - ref) - tol)[~spoilt].max() <= 0


NAN, INF, ALL = float("nan"), float("inf"), slice(None)
SCORES = {"plain": {}, "cap": dict(softcap=20.0), "alibi": dict(alibi=True), "cap_alibi": dict(softcap=20.0, alibi=True)}


@pytest.mark.parametrize("score", list(SCORES))
@pytest.mark.parametrize("Hq,Hkv,D,B", [(8, 2, 128, 16), (4, 1, 64, 32), (14, 2, 128, 8), (3, 3, 64, 16)])
def test_documents(score, Hq, Hkv, D, B):
    """One document's values are NaN or infinite: the others' queries do not notice."""
    lens, qlens = [700, 129, 60], [300, 129, 0]
    starts = [p // 50 * 50 for L, n in zip(lens, qlens) for p in range(L - n, L)]
    c = Case(lens, Hq, Hkv, D, B, qlens=qlens, starts=starts, **SCORES[score])
    check_poisoned(c, [(0, t, ALL, ALL, NAN) for t in range(450, 470)] + [(0, 610, 0, 5, INF), (0, 611, 0, 5, -INF),
                                                                         (1, 3, Hkv - 1, D - 1, -INF), (1, 77, 0, ALL, INF)])


@pytest.mark.parametrize("score", list(SCORES))
def test_later_keys_and_windows(score):
    """A value that only the latest queries see, and one that leaves their window."""
    c = Case([3000, 90], qlens=[200, 90], window=256, prefix=[8, 0], **SCORES[score])
    check_poisoned(c, [(0, 2999, ALL, ALL, NAN), (0, 2650, 1, 17, INF), (1, 80, 0, ALL, NAN), (0, 2860, 0, 3, NAN)])


def test_keys_between_two_queries():
    """Keys that no query of a block sees lie between keys that some see: the later queries' documents begin after their
    own position's block."""
    starts = [0] + [120] * 31
    for opt in SCORES.values():
        c = Case([132], 4, 1, 128, 16, qlens=[32], starts=starts, **opt)
        check_poisoned(c, [])
        pools = c.pools()
        for t in range(101, 120):
            pools["v_cache"][int(c.tables[0][t // 16]), :, t % 16] = NAN if t % 2 else INF
        c.check(run(c, pools))


def test_bad_values_among_many_sequences():
    """Shares of several contexts each, few of them with bad values."""
    r = np.random.default_rng(4)
    lens = [int(x) for x in np.exp(r.uniform(np.log(64), np.log(1500), 64))]
    for opt in (SCORES["cap"], SCORES["alibi"]):
        c = Case(lens, 16, 4, 128, 16, qlens=[5] * 64, **opt)
        check_poisoned(c, [(s, lens[s] - 1 - s % 5, s % 4, ALL if s % 2 else s, NAN) for s in range(0, 64, 7)])


@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("kw", [dict(window=40), dict(starts=[0] * 110 + [3510] * 490), dict(prefix=[3300])],
                         ids=["window", "documents", "prefix"])
def test_many_bad_values_end(value, kw):
    """Every value is NaN or infinite: so is every output, and the call ends as usual."""
    c = Case([4000], 4, 1, 64, 16, qlens=[600], **kw)
    pools = c.pools()
    pools["v_cache"].fill_(value)
    assert not torch.isfinite(run(c, pools)).any()


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 40])
@pytest.mark.parametrize("kind", ["decode", "multi"])
def test_the_widest_window_is_none(kind, window):
    """Also where a call has more queries than the context holds tokens (flagged): those before its first token see
    nothing, the others what they see without a window."""
    c = Case([20, 50, 3], qlens=[60, 50, 35] if kind == "multi" else None)
    pools = c.pools()
    want = run(c, pools)
    c.window = window
    got = run(c, pools)
    assert torch.equal(bits(got), bits(want))
    if kind == "multi":
        assert pkv.read_device_errors(clear=True) == pkv.DEVERR_SEQ_LEN
        assert torch.all(got[:40] == 0) and torch.all(got[40:60].abs().sum(-1) > 0)


@pytest.mark.parametrize("window", [-1, -2 ** 31, -2 ** 32, -2 ** 40])
def test_negative_windows_are_refused(window):
    for qlens in (None, [2, 2]):
        c = Case([40, 40], qlens=qlens, window=0)
        pools = c.pools()
        c.window = window
        with pytest.raises(pkv.PkvError):
            run(c, pools)
