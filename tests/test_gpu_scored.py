"""GPU parity of scored attention (capped or biased scores, windows, documents, prefixes) against the fp64 oracle:
decode over float32, bfloat16 and row-scaled FP8 caches, and several queries a sequence.  Slots that no sequence owns hold
NaN (FP8: NaN codes and scale bytes of 255), so a read of a key that is not seen would show."""
import numpy as np
import pytest
import torch

import paged_kv_cache_279_gb300 as pkv
from paged_kv_cache_279_gb300 import workloads as wl
from harness import bits
from scored_cases import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_errors():
    pkv.read_device_errors(clear=True)
    yield
    assert pkv.read_device_errors(clear=True) == 0


def run(c: Case, pools=None, stream=None, workspace=None, max_seq_len=None, max_q_len=None, out=None, **over):
    pools = c.pools() if pools is None else pools
    args = dict(c.device_args(), workspace=workspace, stream=stream, **over)
    q = c.q.cuda()
    out = torch.full_like(q, float("nan")) if out is None else out
    maxL = max(1, max(c.lens)) if max_seq_len is None else max_seq_len
    if c.qlens is not None:
        pkv.paged_attention_multi_token_scored(out, q, **pools, q_starts=torch.from_numpy(c.q_starts).cuda(), scale=c.scale,
                                               max_q_len=max_q_len or max(1, max(c.qlens)), max_seq_len=maxL, **args)
    elif c.rows:
        pkv.paged_attention_decode_scored_fp8_rows(out, q, **pools, scale=c.scale, max_seq_len=maxL, **args)
    else:
        pkv.paged_attention_decode_scored(out, q, **pools, scale=c.scale, max_seq_len=maxL, **args)
    torch.cuda.synchronize()
    return out


RAGGED = [1, 17, 0, 33, 100, 16, 511, 700, 2, 1300]
OPTIONS = {
    "plain": {},
    "cap": dict(softcap=20.0),
    "tight_cap": dict(softcap=0.5),
    "alibi": dict(alibi=True),
    "window1": dict(window=1),
    "window37": dict(window=37),
    "sinks": dict(window=50, prefix=[4, 0, 3, 40, 100, -5, 4, 600, 9, 1]),
    "starts": dict(starts=[0, 16, 0, 33, 50, 15, 480, 1, -3, 1299]),
    "all": dict(softcap=20.0, alibi=True, window=64, prefix=[1, 2, 3, 20, 90, 16, 300, 10, 2, 700],
                starts=[0, 3, 0, 5, 60, 20, 17, 200, 0, 650]),
}


@pytest.mark.parametrize("kind", ["f32", "bf16", "rows"])
@pytest.mark.parametrize("opt", list(OPTIONS))
def test_decode_options(kind, opt):
    c = Case(RAGGED, dtype=torch.float32 if kind == "f32" else torch.bfloat16, rows=kind == "rows", **OPTIONS[opt])
    c.check(run(c), opt)


@pytest.mark.parametrize("kind", ["f32", "bf16", "rows"])
@pytest.mark.parametrize("Hq,Hkv,D,B", [(1, 1, 64, 16), (3, 1, 128, 32), (10, 2, 64, 32), (32, 4, 128, 16), (7, 7, 128, 16),
                                        (12, 2, 64, 8), (14, 2, 128, 8)])
def test_decode_heads_and_blocks(kind, Hq, Hkv, D, B):
    if kind == "rows" and B == 8:
        pytest.skip("the FP8 caches take blocks of 16 and 32")
    c = Case([5, 64, 31, 257, 1025], Hq, Hkv, D, B, dtype=torch.float32 if kind == "f32" else torch.bfloat16,
             rows=kind == "rows", softcap=15.0, alibi=True, window=200, prefix=[0, 8, 40, 3, 17], seed=3)
    c.check(run(c))


@pytest.mark.parametrize("kind", ["bf16", "rows"])
def test_decode_long_contexts(kind):
    c = Case([4096, 3000, 4001], 8, 2, rows=kind == "rows", softcap=30.0, alibi=True)
    c.check(run(c))
    c = Case([4096, 3000, 4001], 8, 2, rows=kind == "rows", window=1000, prefix=[5, 0, 100])
    c.check(run(c))


def test_decode_many_sequences():
    lens = [(37 * i) % 190 for i in range(300)]
    for rows in (False, True):
        c = Case(lens, 4, 2, 64, 16, softcap=10.0, window=90, rows=rows)
        c.check(run(c, max_seq_len=256))


@pytest.mark.parametrize("kind", ["bf16", "rows"])
def test_decode_thousands_of_sequences(kind):
    """More sequences than the tensor-core kernel's table holds."""
    c = Case([(7 * i) % 23 for i in range(8200)], 2, 1, 64, 16, softcap=10.0, alibi=True, window=11, rows=kind == "rows")
    c.check(run(c))


@pytest.mark.parametrize("Hq,Hkv,D,B", [(1, 1, 64, 16), (8, 1, 128, 32), (6, 2, 64, 8), (7, 7, 128, 16)])
def test_decode_float32_partitions(Hq, Hkv, D, B):
    """Float32 contexts around the sizes at which its kernel splits them, some of whose parts see nothing."""
    c = Case([511, 512, 513, 1024, 1025, 2000], Hq, Hkv, D, B, dtype=torch.float32, softcap=12.0, alibi=True, window=300,
             prefix=[0, 1, 513, 0, 600, 2])
    c.check(run(c))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_decode_append_stores_the_token(kind):
    dt = torch.float32 if kind == "f32" else torch.bfloat16
    for B, D in ((16, 128), (8, 64), (32, 128)):
        c = Case([1, 17, 600, 32, 4], 8, 2, D, B, dtype=dt, softcap=20.0, window=300, prefix=[0, 2, 4, 0, 1])
        want = c.pools()
        pools = c.pools()
        last = [int(c.tables[s][(L - 1) // B]) * B + (L - 1) % B for s, L in enumerate(c.lens)]
        for n in ("k_cache", "v_cache"):
            for x in last:
                pools[n][x // B, :, x % B] = float("nan")
        new = dict(k_new=torch.stack([k[-1] for k in c.ks]).cuda(), v_new=torch.stack([v[-1] for v in c.vs]).cuda())
        c.check(run(c, pools, **new))
        for n in want:
            assert torch.equal(bits(pools[n]), bits(want[n]))


MULTI = [
    dict(lens=[5, 40, 300, 1, 16], qlens=[5, 5, 5, 1, 3]),
    dict(lens=[700, 129, 64], qlens=[300, 129, 1]),
    dict(lens=[1100], qlens=[1100]),
    dict(lens=[257, 0, 33, 500], qlens=[0, 0, 33, 200]),
]


def _multi_options(lens, qlens):
    cum = [0]
    for L, n in zip(lens, qlens):  # documents of 50 tokens
        cum += [((L - n + i) // 50) * 50 for i in range(n)]
    docs = cum[1:]
    late = [(x + 60 if i % 3 == 2 else x) for i, x in enumerate(docs)]
    late = list(np.concatenate([np.maximum.accumulate(np.array(late[a:b], dtype=np.int64)) for a, b in
                                zip(np.cumsum([0] + qlens[:-1]), np.cumsum(qlens)) if b > a]).astype(int)) if docs else []
    return {
        "plain": {},
        "cap": dict(softcap=20.0),
        "alibi": dict(alibi=True),
        "window": dict(window=70),
        "window1": dict(window=1),
        "prefix": dict(prefix=[max(0, L - 3) for L in lens]),
        "all_prefix": dict(prefix=[L + 7 for L in lens]),
        "docs": dict(starts=docs),
        "empty_rows": dict(starts=late),
        "all": dict(softcap=20.0, alibi=True, window=90, prefix=[L // 3 for L in lens], starts=docs),
    }


@pytest.mark.parametrize("shape", range(len(MULTI)))
@pytest.mark.parametrize("opt", ["plain", "cap", "alibi", "window", "window1", "prefix", "all_prefix", "docs", "empty_rows",
                                 "all"])
def test_multi_options(shape, opt):
    m = MULTI[shape]
    c = Case(**m, **_multi_options(m["lens"], m["qlens"])[opt], Hq=8, Hkv=2)
    c.check(run(c), opt)


@pytest.mark.parametrize("Hq,Hkv,D,B", [(1, 1, 64, 16), (3, 1, 128, 32), (10, 2, 64, 32), (16, 2, 128, 16), (5, 5, 128, 8),
                                        (14, 2, 64, 8), (6, 1, 128, 16)])
@pytest.mark.parametrize("qlens", [[5, 3, 1], [200, 90, 333]])
def test_multi_heads_and_blocks(Hq, Hkv, D, B, qlens):
    c = Case([470, 90, 600], Hq, Hkv, D, B, qlens=qlens, softcap=15.0, alibi=True, window=250, prefix=[0, 40, 20], seed=5)
    c.check(run(c))


@pytest.mark.parametrize("opt", [{}, dict(alibi=True), dict(alibi=True, softcap=300.0), dict(softcap=400.0),
                                 dict(alibi=True, prefix=[650, 200, 0, 1500], window=100)],
                         ids=["plain", "alibi", "cap_alibi", "wide_cap", "prefix_alibi"])
@pytest.mark.parametrize("D", [64, 128])
def test_multi_scores_far_apart(opt, D):
    """Scores that differ by hundreds of powers of two, so that the rows' references move within tiles and between them."""
    c = Case([700, 260, 131, 1700], 8, 2, D, 16, qlens=[200, 131, 5, 300], qmul=60.0, **opt)
    assert c.D == D
    c.check(run(c))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("opt", [dict(softcap=30.0), dict(alibi=True), {}], ids=["cap", "alibi", "plain"])
def test_multi_few_queries_of_many_sequences(opt, D):
    """Every SM streams whole contexts of few rows, V behind K: right, and the same bits in every run."""
    r = np.random.default_rng(5)
    c = Case([int(x) for x in np.exp(r.uniform(np.log(64), np.log(2048), 64))], 32, 8, D, 16, qlens=[5] * 64, qmul=1.0, **opt)
    pools = c.pools()
    first = run(c, pools)
    c.check(first)
    for _ in range(5):
        assert torch.equal(bits(run(c, pools)), bits(first))


@pytest.mark.parametrize("kind", ["f32", "bf16", "rows", "multi"])
def test_a_single_key_gives_its_value(kind):
    """A row that sees one key gets that key's value, rounded to the output's type and no more."""
    c = Case([300, 77, 1], 8, 2, qlens=[40, 77, 1] if kind == "multi" else None, window=1, softcap=20.0, rows=kind == "rows",
             dtype=torch.float32 if kind == "f32" else torch.bfloat16)
    got = run(c).float().cpu()
    for s, L in enumerate(c.lens):
        for i in range(int(c.q_starts[s]), int(c.q_starts[s + 1])):
            p = L - int(c.q_starts[s + 1]) + i
            want = c.vs[s][p].repeat_interleave(c.Hq // c.Hkv, 0).to(c.dtype).float()
            tol = 2.0 ** -22 * want.abs() if kind == "f32" else 0.0 * want
            assert bool(((got[i] - want).abs() <= tol).all()), (s, p)


def test_multi_scores_that_grow_and_shrink():
    """Keys whose scores rise, or fall, steadily along the context: every tile has a larger maximum than the one before it."""
    for sign in (1.0, -1.0):
        c = Case([1500, 900], 4, 1, 128, 16, qlens=[140, 33])
        for s, L in enumerate(c.lens):
            ramp = torch.linspace(0.0, 2.0 * sign, L)[:, None, None]
            c.ks[s] = (ramp + 0.01 * c.ks[s].float()).to(torch.bfloat16)
        c.q = (c.q.float().abs() + 1.0).to(torch.bfloat16)
        c.check(run(c), f"sign {sign}")


def test_one_query_per_sequence_is_the_decode():
    lens = [1, 17, 33, 100, 511, 700, 1300]
    a = Case(lens, softcap=20.0, alibi=True, window=300)
    b = Case(lens, qlens=[1] * 7, softcap=20.0, alibi=True, window=300)
    a.check(run(b))
    assert (run(a).float() - run(b).float()).abs().max() < 2.0 ** -5  # both within their bounds; outputs below 4


@pytest.mark.parametrize("kind", ["f32", "bf16", "rows", "multi"])
def test_borders_are_exact(kind):
    """A key just outside the window, the document or the prefix carries a score that would swamp every other; the keys
    just inside carry the next largest ones, so the result is theirs."""
    W, L, start, pre = 40, 333, 0, 7
    c = Case([L], 2, 1, 64, 16, qlens=[1] if kind == "multi" else None, window=W, prefix=[pre],
             dtype=torch.float32 if kind == "f32" else torch.bfloat16, rows=False, qmul=0.0, scale=1.0)
    c.q[:] = 0
    c.q[..., 0] = 1.0
    p = L - 1
    for hot, seen in ((p - W, False), (p - W + 1, True), (pre, False), (pre - 1, True), (p, True)):
        k = torch.zeros(L, 1, 64)
        k[hot, 0, 0] = 64.0
        v = torch.full((L, 1, 64), -1.0)
        v[hot] = 1.0
        c.ks, c.vs = [k.to(c.dtype)], [v.to(c.dtype)]
        if kind == "rows":
            from oracle import fp8_rows
            c.rows = True
            c.codes = [(fp8_rows.quantise_rows(k.numpy()), fp8_rows.quantise_rows(v.numpy()))]
        out = run(c)
        # exp(-64) of the other keys' weight is below every rounding; a mean of L equal values is off by at most the
        # roundings of two sums of L terms
        near = lambda x, y: bool(((x.float() - y).abs() <= L * 2.0 ** -23).all())  # noqa: E731
        assert near(out, 1.0 if seen else -1.0), (hot, out.unique())
        c.starts, c.window = [hot + 1], 0
        assert torch.all(run(c) == 0.0) if hot == p else near(run(c), -1.0)
        c.starts = [hot]
        assert near(run(c), 1.0)
        c.starts, c.window = None, W


@pytest.mark.parametrize("kind", ["f32", "bf16", "rows"])
def test_decode_values_of_one_token(kind):
    c = Case([1, 1, 9], dtype=torch.float32 if kind == "f32" else torch.bfloat16, rows=kind == "rows", softcap=5.0,
             alibi=True, window=1)
    out = run(c)
    rep = c.Hq // c.Hkv
    for s, L in enumerate(c.lens):  # one key seen: its V row itself
        assert torch.equal(out[s].double().cpu(), c.vs[s][L - 1].double().repeat_interleave(rep, 0))


@pytest.mark.parametrize("kind", ["f32", "bf16", "rows", "multi"])
def test_nan_and_infinity_in_hidden_places_do_not_show(kind):
    lens = [300, 64]
    c = Case(lens, qlens=[3, 2] if kind == "multi" else None, dtype=torch.float32 if kind == "f32" else torch.bfloat16,
             rows=kind == "rows", window=30, prefix=[5, 0])
    pools = c.pools()
    hidden = {0: range(6, 260), 1: range(0, 30)}  # seen by no query of either form
    for s, r in hidden.items():
        for t in r:
            blk, off = int(c.tables[s][t // 16]), t % 16
            if kind == "rows":
                pools["k_cache"][blk, :, off], pools["v_cache"][blk, :, off] = 0x7F, 0xFF
                pools["k_scales"][blk, :, off], pools["v_scales"][blk, :, off] = 255, 255
            else:
                pools["k_cache"][blk, :, off] = float("inf") if t % 2 else float("nan")
                pools["v_cache"][blk, :, off] = float("-inf") if t % 3 else float("nan")
    c.check(run(c, pools))


@pytest.mark.parametrize("kind", ["f32", "bf16", "rows", "multi"])
def test_nan_in_a_seen_place_shows(kind):
    c = Case([40, 40], qlens=[2, 2] if kind == "multi" else None, rows=kind == "rows",
             dtype=torch.float32 if kind == "f32" else torch.bfloat16)
    pools = c.pools()
    blk = int(c.tables[1][0])
    pools["v_cache"][blk, :, 3, 7] = 0x7F if kind == "rows" else float("nan")
    out = run(c, pools)
    a, b = int(c.q_starts[1]), int(c.q_starts[2])
    assert torch.isnan(out[a:b, :, 7]).all() and torch.isfinite(out[:a]).all()
    pools = c.pools()
    pools["k_cache"][blk, :, 3, 7] = 0x7F if kind == "rows" else float("nan")
    out = run(c, pools)
    assert torch.isnan(out[a:b]).all() and torch.isfinite(out[:a]).all()


@pytest.mark.parametrize("kind", ["bf16", "rows", "multi"])
def test_placement_does_not_matter(kind):
    kw = dict(qlens=[200, 7] if kind == "multi" else None, rows=kind == "rows", softcap=20.0, window=500, prefix=[30, 0])
    a = Case([900, 450], **kw)
    x = run(a)
    perm = np.random.default_rng(3).permutation(a.NB)
    a.tables = np.where(a.tables >= 0, perm[np.maximum(a.tables, 0)], -1).astype(np.int32)
    assert torch.equal(bits(x), bits(run(a)))


@pytest.mark.parametrize("scale", [0.0, -0.1])
@pytest.mark.parametrize("kind", ["f32", "bf16", "rows", "multi"])
def test_any_finite_scale(kind, scale):
    c = Case([77, 300], qlens=[9, 130] if kind == "multi" else None, rows=kind == "rows", scale=scale, softcap=9.0,
             dtype=torch.float32 if kind == "f32" else torch.bfloat16)
    c.check(run(c))


@pytest.mark.parametrize("cap", [60.0, 1e3, 1e6, 3e38])
@pytest.mark.parametrize("kind", ["f32", "bf16", "rows", "multi"])
def test_wide_caps_cost_no_accuracy(kind, cap):
    """Scores far below their cap: the bound is the uncapped one, plus 2^-19 of a score (z >= 1/4: 2^-21 of the cap, at most
    four times the score; below it the series' 2^-21 and its arithmetic)."""
    c = Case([77, 300], qlens=[9, 130] if kind == "multi" else None, rows=kind == "rows", softcap=cap, window=90,
             dtype=torch.float32 if kind == "f32" else torch.bfloat16)
    got = run(c).double().cpu().numpy()
    ref, _ = c.reference()
    c.softcap = 0.0
    _, tol = c.reference()
    rep, at = c.Hq // c.Hkv, 0
    for s, L in enumerate(c.lens):
        n = int(c.q_starts[s + 1] - c.q_starts[s])
        q, k = (x.double().abs().numpy() for x in (c.q[at:at + n], c.ks[s]))
        a = c.scale * max(float((q[:, h] @ k[:, h // rep].T).max()) for h in range(c.Hq))
        tol[at:at + n] += 4 * 2.0 ** -19 * a * c.vs[s].double().abs().max().item()
        at += n
    assert np.all(np.abs(got - ref) <= tol)


@pytest.mark.parametrize("kind", ["f32", "bf16", "rows", "multi"])
def test_negative_and_large_slopes(kind):
    c = Case([200, 1000], qlens=[9, 150] if kind == "multi" else None, rows=kind == "rows", alibi=True,
             dtype=torch.float32 if kind == "f32" else torch.bfloat16)
    c.slopes = np.array([3.0, -0.02, 0.5, -0.3, 40.0, 0.0, 0.001, 7.0], np.float32)
    c.check(run(c))


def test_rows_of_extreme_scales():
    """V rows whose sizes differ by 2^60, the small ones carrying all the weight: nothing is lost."""
    c = Case([200], 2, 1, rows=True)
    from oracle import fp8_rows
    r = np.random.default_rng(11)
    k, v = r.standard_normal((200, 1, 128)).astype(np.float32), r.standard_normal((200, 1, 128)).astype(np.float32)
    v[::2] *= 2.0 ** 30
    v[1::2] *= 2.0 ** -30
    k[::2] = -3.0 * c.q[0, :1].float().numpy()   # large rows: scores far below the others'
    k[1::2] *= 0.1
    c.codes = [(fp8_rows.quantise_rows(k), fp8_rows.quantise_rows(v))]
    c.ks, c.vs = ([torch.from_numpy(fp8_rows.row_values(*p))] for p in c.codes[0])
    c.window = 1                                  # the last token, a small row
    c.check(run(c))
    c.window, c.softcap = 0, 0.0
    c.q = c.q[:, :1].repeat(1, 2, 1)
    ref, tol = c.reference()
    g = run(c).double().cpu().numpy()
    assert np.all(np.abs(g - ref) <= tol)


@pytest.mark.parametrize("kind", ["f32", "bf16", "rows", "multi", "append"])
def test_captured_and_replayed(kind):
    """One call in a CUDA graph over a workspace of random bytes, replayed with queries, lengths and windows' places
    refreshed in place."""
    lens = [700, 90, 1300]
    c = Case(lens, qlens=[150, 90, 7] if kind == "multi" else None, rows=kind == "rows", softcap=20.0, window=400,
             dtype=torch.float32 if kind == "f32" else torch.bfloat16)
    pools = c.pools()
    new = dict(k_new=torch.stack([k[-1] for k in c.ks]).cuda(), v_new=torch.stack([v[-1] for v in c.vs]).cuda()) \
        if kind == "append" else {}
    S, T = len(lens), c.q.shape[0]
    need = (pkv.paged_attention_multi_token_scored_workspace_size(T, c.Hq, c.D, 1300) if kind == "multi" else
            pkv.paged_attention_decode_scored_workspace_size(S, c.Hq, c.D, 1300))
    ws = torch.randint(0, 256, (max(need, 1),), dtype=torch.uint8, device="cuda")
    q = c.q.cuda()
    out = torch.full_like(q, float("nan"))
    args = c.device_args()
    call = dict(pools, **args, workspace=ws, scale=c.scale, max_seq_len=1300, **new)

    def go():
        if kind == "multi":
            pkv.paged_attention_multi_token_scored(out, q, q_starts=q_starts, max_q_len=150, **call)
        elif kind == "rows":
            pkv.paged_attention_decode_scored_fp8_rows(out, q, **call)
        else:
            pkv.paged_attention_decode_scored(out, q, **call)
    q_starts = torch.from_numpy(c.q_starts).cuda()
    go()  # first use outside the capture
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            go()
    torch.cuda.current_stream().wait_stream(s)
    for it in range(3):
        c.q = torch.roll(c.q, 1, 0)
        q.copy_(c.q)
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        c.check(out, f"replay {it}")


@pytest.mark.parametrize("kind", ["f32", "bf16", "rows", "multi"])
def test_captured_without_a_workspace(kind):
    """The call's own workspace inside a CUDA graph, beside eager calls and allocations on the stream of the replays."""
    c = Case([900, 33, 1200], qlens=[60, 3, 9] if kind == "multi" else None, rows=kind == "rows", softcap=15.0, alibi=True,
             dtype=torch.float32 if kind == "f32" else torch.bfloat16)
    pools = c.pools()
    want = run(c, pools)
    q, out, args = c.q.cuda(), torch.full_like(want, float("nan")), c.device_args()
    f = (pkv.paged_attention_multi_token_scored if kind == "multi" else
         pkv.paged_attention_decode_scored_fp8_rows if c.rows else pkv.paged_attention_decode_scored)
    call = dict(pools, **args, scale=c.scale, max_seq_len=1200,
                **(dict(q_starts=torch.from_numpy(c.q_starts).cuda(), max_q_len=60) if kind == "multi" else {}))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        f(out, q, **call)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for _ in range(2):
                f(out, q, **call)
        for _ in range(3):
            out.fill_(float("nan"))
            junk = torch.randn(1 << 22, device="cuda")
            g.replay()
            again = f(torch.empty_like(out), q, **call)
            junk.mul_(2.0)
            assert torch.equal(bits(out), bits(want)) and torch.equal(bits(again), bits(want))
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind", ["bf16", "rows", "multi"])
def test_two_calls_on_two_streams(kind):
    kw = dict(qlens=[150, 90, 7] if kind == "multi" else None, rows=kind == "rows", softcap=20.0)
    a, b = Case([700, 90, 1300], **kw), Case([600, 95, 1000], seed=9, **kw)
    pa, pb = a.pools(), b.pools()
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    oa = run(a, pa, stream=sa)
    ob = run(b, pb, stream=sb.cuda_stream)
    a.check(oa)
    b.check(ob)


def test_max_seq_len_zero_gives_zeros():
    c = Case([0, 0], rows=False)
    assert torch.all(run(c, max_seq_len=0) == 0)
    c = Case([0, 0], rows=True)
    assert torch.all(run(c, max_seq_len=0) == 0)


@pytest.mark.parametrize("kind", ["f32", "bf16", "rows", "multi"])
def test_bad_blocks_and_lengths_are_flagged(kind):
    c = Case([100, 100], qlens=[2, 2] if kind == "multi" else None, rows=kind == "rows",
             dtype=torch.float32 if kind == "f32" else torch.bfloat16)
    good, pools = c.tables.copy(), c.pools()
    c.tables[0, 2] = c.NB + 5
    out = run(c, pools)
    assert pkv.read_device_errors(clear=True) == pkv.DEVERR_BLOCK_ID
    assert torch.isfinite(out).all()
    # a bad id where no query looks is not an error
    c.tables = good.copy()
    c.tables[0, 0] = -7
    c.window = 20
    ref = run(c, pools)
    c.tables = good
    assert torch.equal(bits(ref), bits(run(c, pools)))
    assert pkv.read_device_errors(clear=True) == 0
    c.window = 0
    c.lens = [-1, 100]
    out = run(c, pools, max_seq_len=100)
    assert pkv.read_device_errors(clear=True) == pkv.DEVERR_SEQ_LEN
    a = int(c.q_starts[1])
    assert torch.all(out[:a] == 0) and torch.isfinite(out).all()
    c.lens = [101 * 16, 100]  # above what the table holds
    out = run(c, pools, max_seq_len=2000)
    assert pkv.read_device_errors(clear=True) & pkv.DEVERR_SEQ_LEN


def test_multi_bad_query_ranges_are_flagged():
    c = Case([100, 100, 100], qlens=[4, 4, 4])
    q, pools = c.q.cuda(), c.pools()
    args = dict(c.device_args(), scale=c.scale, max_q_len=4, max_seq_len=100)
    for starts, bits_ in (([0, 8, 4, 12], pkv.DEVERR_SEQ_LEN), ([0, 4, 8, 13], pkv.DEVERR_SEQ_LEN),
                          ([-2, 4, 8, 12], pkv.DEVERR_SEQ_LEN)):
        out = torch.full_like(q, 7.0)
        pkv.paged_attention_multi_token_scored(out, q, **pools, q_starts=torch.tensor(starts, dtype=torch.int32).cuda(), **args)
        assert pkv.read_device_errors(clear=True) == bits_
        assert torch.isfinite(out).all()
    # more queries than max_q_len: the rest of the rows stay as they were
    out = torch.full_like(q, 7.0)
    args["max_q_len"] = 3
    pkv.paged_attention_multi_token_scored(out, q, **pools, q_starts=torch.from_numpy(c.q_starts).cuda(), **args)
    assert pkv.read_device_errors(clear=True) == pkv.DEVERR_SEQ_LEN
    assert torch.all(out[3] == 7.0) and torch.all(out[7] == 7.0) and not torch.any(out[0] == 7.0)
    # more queries than the context holds: those before its first token see nothing
    c = Case([3, 50], qlens=[5, 2], softcap=10.0)
    out = run(c)
    assert pkv.read_device_errors(clear=True) == pkv.DEVERR_SEQ_LEN
    assert torch.all(out[:2] == 0) and torch.isfinite(out).all()
    # a prefix they all see
    c.prefix = [2, 0]
    out = run(c)
    assert pkv.read_device_errors(clear=True) == pkv.DEVERR_SEQ_LEN
    assert torch.all(out[:2].abs().sum(-1) > 0)


def test_rows_behind_the_last_sequence_are_left():
    c = Case([60, 70], qlens=[3, 140])
    c.lens = [60, 140]
    c = Case([60, 140], qlens=[3, 140])
    q = torch.cat([c.q, c.q[:9]]).cuda()
    out = torch.full_like(q, 5.0)
    pkv.paged_attention_multi_token_scored(out, q, **c.pools(), **c.device_args(), scale=c.scale, max_q_len=140,
                                           max_seq_len=140, q_starts=torch.from_numpy(c.q_starts).cuda())
    torch.cuda.synchronize()
    assert torch.all(out[143:] == 5.0)
    c.check(out[:143])


def test_serving_run_over_the_quantised_cache():
    """A prompt is quantised as it is written; its values are read back into a bf16 pool and prefilled in chunks; then
    tokens are appended and decoded over the quantised cache, against the oracle over the cache's own values."""
    from oracle import fp8_rows
    from oracle.scored import scored_attention
    Hq, Hkv, D, B, L0, steps = 8, 2, 128, 16, 75, 3
    alloc = pkv.BlockAllocator(32, B)
    assert alloc.add_seq(0, L0) == 0
    r = np.random.default_rng(2)
    bf = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32)).to(torch.bfloat16)  # noqa: E731
    k, v, q = bf(L0 + steps, Hkv, D), bf(L0 + steps, Hkv, D), bf(L0 + steps, Hq, D)
    codes = {n: torch.full((32, Hkv, B, D), 0xFF, dtype=torch.uint8, device="cuda") for n in "kv"}
    scales = {n: torch.full((32, Hkv, B), 0xFF, dtype=torch.uint8, device="cuda") for n in "kv"}
    pool = {n: torch.full((32, Hkv, B, D), float("nan"), dtype=torch.bfloat16, device="cuda") for n in "kv"}
    slots = torch.from_numpy(alloc.slots(0, 0, L0)).cuda()
    pkv.kv_cache_write_fp8_rows(k[:L0].cuda(), v[:L0].cuda(), codes["k"], codes["v"], scales["k"], scales["v"], slots)
    kb, vb = torch.empty(L0, Hkv, D, dtype=torch.bfloat16, device="cuda"), torch.empty(L0, Hkv, D, dtype=torch.bfloat16, device="cuda")
    pkv.kv_cache_read_fp8_rows(kb, vb, codes["k"], codes["v"], scales["k"], scales["v"], slots)
    pkv.kv_cache_write(kb, vb, pool["k"], pool["v"], slots)
    kv = [fp8_rows.row_values(*fp8_rows.quantise_rows(x.float().numpy())) for x in (k, v)]
    opts = dict(softcap=12.0, window=50)
    out = torch.empty(L0, Hq, D, dtype=torch.bfloat16, device="cuda")
    for a, b in ((0, 32), (32, 75)):
        tables, lens = alloc.block_tables([0], cap=8)
        pkv.paged_attention_multi_token_scored(
            out[a:b], q[a:b].cuda(), pool["k"], pool["v"], torch.from_numpy(tables).cuda(),
            torch.tensor([b], dtype=torch.int32, device="cuda"), torch.tensor([0, b - a], dtype=torch.int32, device="cuda"),
            0.09, 64, 128, **opts)
    ref, size = scored_attention(q[:L0].float().numpy(), kv[0][:L0], kv[1][:L0], 0.09, **opts)
    err = np.abs(out.double().cpu().numpy() - ref)
    assert np.all(err <= 2.0 ** -8 * np.abs(ref) + 2 * (2.0 ** -8 + 2.0 ** -12) * size)
    for i in range(steps):
        st, slot, pairs = alloc.append_slots([0])
        assert st == 0 and len(pairs) == 0
        n = L0 + i + 1
        pkv.kv_cache_write_fp8_rows(k[n - 1:n].cuda(), v[n - 1:n].cuda(), codes["k"], codes["v"], scales["k"], scales["v"],
                                    torch.from_numpy(np.asarray(slot)).cuda())
        tables, lens = alloc.block_tables([0], cap=8)
        o = torch.empty(1, Hq, D, dtype=torch.bfloat16, device="cuda")
        pkv.paged_attention_decode_scored_fp8_rows(o, q[n - 1:n].cuda(), codes["k"], codes["v"], scales["k"], scales["v"],
                                                   torch.from_numpy(tables).cuda(), torch.from_numpy(lens).cuda(), 0.09, 128,
                                                   **opts)
        ref, size = scored_attention(q[n - 1:n].float().numpy(), kv[0][:n], kv[1][:n], 0.09, **opts)
        err = np.abs(o.double().cpu().numpy() - ref)
        assert np.all(err <= 2.0 ** -8 * np.abs(ref) + 2 * (2.0 ** -8 + 2.0 ** -12) * size)
    torch.cuda.synchronize()


def test_arguments_are_refused():
    c = Case([40, 40])
    pools, args = c.pools(), c.device_args()
    q = c.q.cuda()
    out = torch.empty_like(q)
    call = dict(pools, **args, scale=c.scale, max_seq_len=40)
    f = pkv.paged_attention_decode_scored
    with pytest.raises(pkv.PkvError):
        f(out, q, **dict(call, softcap=-1.0))
    with pytest.raises(pkv.PkvError):
        f(out, q, **dict(call, softcap=float("inf")))
    with pytest.raises(pkv.PkvError):
        f(out, q, **dict(call, window=-1))
    with pytest.raises(pkv.PkvError):
        f(out, q, **dict(call, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"), max_seq_len=4000))
    with pytest.raises(ValueError):
        f(out, q, **dict(call, alibi_slopes=torch.zeros(3, device="cuda")))
    with pytest.raises(TypeError):
        f(out, q, **dict(call, alibi_slopes=torch.zeros(8, device="cuda", dtype=torch.float64)))
    with pytest.raises(ValueError):
        f(out, q, **dict(call, prefix_lens=torch.zeros(3, device="cuda", dtype=torch.int32)))
    with pytest.raises(ValueError):
        f(out, q, **dict(call, key_starts=torch.zeros(1, device="cuda", dtype=torch.int32)))
    with pytest.raises(TypeError):
        f(out, q, **dict(call, seq_lens=torch.tensor([40, 40], dtype=torch.int32)))
    with pytest.raises(ValueError):
        f(out.transpose(0, 1).contiguous().transpose(0, 1), q, **call)
    with pytest.raises(TypeError):
        f(out, q.half(), **call)
    with pytest.raises(ValueError):
        f(out, q, **dict(call, k_new=torch.zeros(2, 2, 128, device="cuda", dtype=torch.bfloat16)))
    with pytest.raises(TypeError):
        pkv.paged_attention_multi_token_scored(out.float(), q.float(), **call, q_starts=torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"), max_q_len=1)
