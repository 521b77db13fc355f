"""GPU: attention over a paged cache of latent rows, against the fp64 oracle."""
import numpy as np
import pytest
import torch

import latent_cases as lc
import paged_kv_cache_279_gb300 as pkv
from oracle import rotary

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _clear_errors():
    pkv.read_device_errors(clear=True)
    yield
    assert pkv.read_device_errors(clear=True) == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens,H,V,B", [([1, 17, 33, 100], 4, 512, 16), ([1], 1, 256, 8), ([64], 16, 512, 64), ([65, 63, 128], 3, 256, 32),
                                        ([129, 1, 700], 33, 512, 16), ([1500], 64, 512, 32), ([40] * 9, 65, 256, 16),
                                        ([300, 2], 128, 512, 8), ([2000] + [5] * 30, 20, 512, 16)])
def test_decode(dtype, lens, H, V, B):
    c = lc.make(lens, H, V, B, dtype)
    lc.check(lc.run(c), c)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens,nq,H,V,B", [([7], [7], 4, 512, 16), ([100, 33, 1], [5, 1, 1], 16, 512, 16), ([200], [130], 3, 256, 8),
                                           ([64, 65], [64, 65], 1, 512, 64), ([300, 40], [9, 40], 33, 256, 32),
                                           ([90, 500], [64, 3], 128, 512, 16), ([20, 30, 40], [0, 5, 0], 16, 512, 16)])
def test_multi_token(dtype, lens, nq, H, V, B):
    c = lc.make(lens, H, V, B, dtype, queries=nq)
    lc.check(lc.run(c), c)


FAR = 10 ** 6  # a limit above the contexts: they are cut into shares and joined, however short


@pytest.mark.parametrize("lens,H,V,B", [([1, 17, 33, 100], 4, 512, 16), ([64], 16, 512, 64), ([65, 63, 128], 3, 256, 32), ([0, 129, 0, 1, 700], 33, 512, 16),
                                        ([40] * 9, 65, 256, 16), ([300, 2, 0], 128, 512, 8), ([130] * 170, 10, 256, 8)])
def test_decode_cut(lens, H, V, B):
    c = lc.make(lens, H, V, B)
    lc.check(lc.run(c, max_len=FAR), c)


@pytest.mark.parametrize("lens,nq,H,V,B", [([7], [7], 4, 512, 16), ([100, 33, 1], [5, 1, 1], 4, 512, 16), ([200], [130], 3, 256, 8),
                                           ([64, 65], [64, 65], 1, 512, 64), ([300, 40], [9, 40], 33, 256, 32), ([90, 500], [64, 3], 128, 512, 16),
                                           ([20, 30, 40], [0, 5, 0], 16, 512, 16), ([33] * 120, [1, 2, 0, 4] * 30, 16, 512, 16)])
def test_multi_token_cut(lens, nq, H, V, B):
    c = lc.make(lens, H, V, B, queries=nq)
    lc.check(lc.run(c, max_len=FAR), c)


def test_long_context_is_split_and_joined():
    for dtype, H in ((BF, 16), (F32, 2), (BF, 2)):
        c = lc.make([9000, 10], H, 512, 16, dtype, seed=3)
        lc.check(lc.run(c), c)


def test_limits_above_the_contexts():
    c = lc.make([50, 90], 16)
    want = lc.run(c)
    got = lc.run(c, max_len=10 ** 9)
    lc.check(got, c)
    lc.check(want, c)
    c = lc.make([50, 90], 16, queries=[3, 4])
    lc.check(lc.run(c, max_len=10 ** 9, max_q=10 ** 9), c)


def test_a_loose_limit_on_the_queries_of_few_rows():
    """Fewer than 64 query rows in all, whatever max_q_len says: the workspace is sized by what there is."""
    for nq, H in (([3], 16), ([2, 1], 1), ([2, 2], 16), ([1], 32)):
        c = lc.make([400, 90][:len(nq)], H, queries=nq)
        n = pkv.paged_latent_attention_workspace_size(sum(nq), H, 512, 400)
        ws = torch.full((n + 4096,), 77, dtype=torch.uint8, device="cuda")
        lc.check(lc.run(c, max_q=10 ** 9, workspace=ws[:n]), c)
        assert torch.all(ws[n:] == 77)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("queries", [None, [2, 3]])
def test_no_tokens_at_all(dtype, queries):
    c = lc.make([8, 8], 5, 256, 8, dtype, queries=queries)
    c["lens"] = [0, 0]
    out = torch.full((c["q"].shape[0] + 1, 5, 256), 7.0, dtype=dtype, device="cuda")
    args = [out[:-1], c["q"].cuda(), c["cache"].cuda(), torch.from_numpy(c["tables"]).cuda(), torch.zeros(2, dtype=torch.int32).cuda()]
    for max_len in (0, 8):
        out.fill_(7.0)
        if queries is None:
            pkv.paged_latent_attention_decode(*args, 0.1, max_len)
        else:
            pkv.paged_latent_attention_multi_token(*args, torch.from_numpy(c["starts"]).cuda(), 0.1, 3, max_len)
        assert torch.all(out[:-1] == 0) and torch.all(out[-1] == 7.0)
    # queries without tokens to stand at are flagged, as are lengths above max_seq_len
    assert pkv.read_device_errors(clear=True) == (pkv.DEVERR_SEQ_LEN if queries else 0)


@pytest.mark.parametrize("V,H", [(512, 4), (256, 20), (512, 100)])
def test_many_sequences(V, H):
    r = np.random.default_rng(0)
    lens = [int(x) for x in r.integers(1, 200, 400)]
    lens[7] = lens[333] = 0
    c = lc.make(lens, H, V, 16, seed=2)
    lc.check(lc.run(c), c)
    lens = [int(x) for x in r.integers(1, 100, 250)]
    c = lc.make(lens, H, V, 32, queries=[int(min(L, x)) for L, x in zip(lens, r.integers(0, 6, 250))], seed=2)
    lc.check(lc.run(c), c)


@pytest.mark.parametrize("V,H,L", [(512, 128, 5000), (256, 128, 3000), (256, 64, 5000), (512, 33, 4000), (256, 8, 7000)])
def test_one_long_context(V, H, L):
    c = lc.make([L], H, V, 64, seed=5)
    lc.check(lc.run(c), c)
    c = lc.make([L, 30], H, V, 16, queries=[5, 2], seed=6)
    lc.check(lc.run(c), c)


def test_empty_contexts_and_rows_of_no_query():
    c = lc.make([0, 30, 0], 5)
    out = lc.run(c)
    assert torch.all(out[[0, 2]] == 0)
    lc.check(out, c)
    c = lc.make([30, 12], 5, queries=[4, 2])
    out = torch.full((9, 5, 512), 7.0, dtype=BF, device="cuda")
    c["q"] = torch.cat([c["q"], torch.full((3, 5, 576), float("nan"), dtype=BF)])
    lc.run(c, out=out)
    assert torch.all(out[6:] == 7.0)
    c["q"] = c["q"][:6]
    lc.check(out[:6], c)


@pytest.mark.parametrize("L,more,H", [(3, 2, 4), (3, 40, 4), (60, 70, 16), (700, 100, 5), (0, 50, 16), (0, 3, 2)])
@pytest.mark.parametrize("max_len", [None, FAR])
def test_more_queries_than_tokens(L, more, H, max_len):
    c = lc.make([L, 40], H, queries=[L, 4])
    # more queries in front of the first sequence's: they see nothing
    r = torch.from_numpy(np.random.default_rng(8).standard_normal((more, H, 576)).astype(np.float32)).to(BF)
    c["q"] = torch.cat([r, c["q"]])
    c["starts"] = np.array([0, L + more, L + more + 4], dtype=np.int32)
    c["nq"] = [L + more, 4]
    out = lc.run(c, max_len=max_len)
    assert pkv.read_device_errors(clear=True) == pkv.DEVERR_SEQ_LEN
    assert torch.all(out[:more] == 0)
    lc.check(out, c)


@pytest.mark.parametrize("queries", [None, [5, 3], [50, 70]])
@pytest.mark.parametrize("dtype,max_len", [(BF, None), (F32, None), (BF, FAR)])
def test_what_is_not_seen_does_not_matter(dtype, max_len, queries):
    """Other slots of the pool hold NaN, infinities, the largest and the lowest numbers: the same bits."""
    c = lc.make([77, 130], 6, 512, 16, dtype, queries, fill=0.0)
    want = lc.run(c, max_len=max_len)
    for fill in (float("nan"), float("inf"), -float("inf"), torch.finfo(dtype).max, torch.finfo(dtype).min):
        d = lc.make([77, 130], 6, 512, 16, dtype, queries, fill=fill)
        assert torch.equal(lc.run(d, max_len=max_len), want)


@pytest.mark.parametrize("dtype,max_len", [(BF, None), (F32, None), (BF, FAR)])
@pytest.mark.parametrize("H", [1, 16, 40])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_bad_row_reaches_only_the_queries_that_see_it(dtype, max_len, H, bad):
    c = lc.make([70, 150, 20], H, 512, 16, dtype, queries=[10, 80, 20])
    want = lc.run(c, max_len=max_len)
    pos, s = 110, 1  # token 110 of sequence 1, whose queries stand at 70 .. 149
    cache = c["cache"].clone()
    cache[int(c["tables"][s][pos // 16]), pos % 16, 33] = bad
    got = lc.run(c, cache=cache.cuda(), max_len=max_len)
    first = c["starts"][s] + (pos - 70)
    keep = torch.ones(110, dtype=torch.bool)
    keep[first:c["starts"][s + 1]] = False
    assert torch.equal(got[keep.cuda()], want[keep.cuda()])
    seen = got[~keep.cuda()].float()
    assert torch.all(~torch.isfinite(seen[..., 33]))


@pytest.mark.parametrize("max_len", [None, FAR])
def test_a_bad_query_stays_by_itself(max_len):
    for queries in (None, [20, 30], [2, 2]):
        c = lc.make([70, 150], 16, queries=queries)
        want = lc.run(c, max_len=max_len)
        c["q"][1, 3] = float("nan")
        got = lc.run(c, max_len=max_len)
        assert torch.all(torch.isnan(got[1, 3]))
        got[1, 3] = want[1, 3]
        assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size", [0.0, 30.0, 1e4])
def test_scores_of_any_size(dtype, size):
    for queries in (None, [40, 3]):
        c = lc.make([150, 600], 9, 512, 16, dtype, queries, size=size)
        lc.check(lc.run(c), c)
        lc.check(lc.run(c, max_len=FAR), c)
        lc.check(lc.run(c, scale=-0.1), c, scale=-0.1)
        lc.check(lc.run(c, scale=0.0), c, scale=0.0)


def test_rising_and_falling_scores():
    """The running maximum moves in every tile, or not after the first."""
    for rising in (False, True):
        c = lc.make([1000], 16, fill=0.0)
        ramp = torch.linspace(-1, 1, 1000) * (400 if rising else -400)
        c["rows"][0][:, 575] = ramp.to(BF)
        c["q"][:, :, 575] = 1.0
        p = np.arange(1000)
        c["cache"][torch.from_numpy(c["tables"][0][p // 16].astype(np.int64)), torch.from_numpy(p % 16)] = c["rows"][0]
        lc.check(lc.run(c, scale=1.0), c, scale=1.0)


def test_placement_does_not_matter():
    a = lc.make([300, 77, 64], 16, queries=[7, 77, 1])
    want = lc.run(a)
    NB = a["cache"].shape[0]
    perm = np.random.default_rng(9).permutation(NB)
    b = dict(a, cache=a["cache"][torch.from_numpy(np.argsort(perm))], tables=perm[a["tables"]].astype(np.int32))
    assert torch.equal(lc.run(b), want)
    assert torch.equal(lc.run(a), want)


def test_bad_blocks_and_lengths():
    c = lc.make([100, 64], 16)
    want = lc.run(c)
    c["tables"] = c["tables"].copy()
    for bad in (-1, c["cache"].shape[0], 2 ** 31 - 1, -2 ** 31):
        t = c["tables"].copy()
        t[0, 2] = bad  # tokens 32 .. 47 are left out
        d = dict(c, tables=t)
        got = lc.run(d)
        assert pkv.read_device_errors(clear=True) == pkv.DEVERR_BLOCK_ID
        e = dict(c, rows=[torch.cat([c["rows"][0][:32], c["rows"][0][48:]]), c["rows"][1]])
        lc.check(got, e)
        assert torch.equal(got[1], want[1])
    for L, cut in ((-3, 0), (200, 112), (2 ** 31 - 1, 112)):
        d = dict(c, lens=[L, 64])
        got = lc.run(d, max_len=5000)
        assert pkv.read_device_errors(clear=True) == pkv.DEVERR_SEQ_LEN
        assert torch.equal(got[1], want[1])
        if cut == 0:
            assert torch.all(got[0] == 0)


def test_bad_query_starts():
    c = lc.make([100, 64, 30], 16, queries=[4, 4, 4])
    want = lc.run(c)
    for starts in ([0, 4, 100, 12], [0, 4, -1, 12]):
        out = lc.run(dict(c, starts=np.array(starts, dtype=np.int32)))
        assert pkv.read_device_errors(clear=True) & pkv.DEVERR_SEQ_LEN
        assert torch.equal(out[:4], want[:4])
    out = lc.run(c, max_q=3)  # queries past max_q are not attended
    assert pkv.read_device_errors(clear=True) == pkv.DEVERR_SEQ_LEN
    keep = torch.tensor([True, True, True, False] * 3).cuda()
    assert torch.all(out[~keep] == 7.0) and torch.equal(out[keep], want[keep])


def test_streams_workspaces_and_graphs():
    c = lc.make([3000, 10, 500], 16)
    want = lc.run(c)
    n = pkv.paged_latent_attention_workspace_size(3, 16, 512, 3000)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN everywhere
    assert torch.equal(lc.run(c, workspace=ws), want)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = lc.run(c, stream=st)
    assert torch.equal(got, want)
    cache, q = c["cache"].cuda(), c["q"].cuda()
    tables, lens = torch.from_numpy(c["tables"]).cuda(), torch.tensor(c["lens"], dtype=torch.int32).cuda()
    outs = [torch.zeros_like(want) for _ in range(2)]
    graphs = []
    for o in outs:  # two graphs that share a workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkv.paged_latent_attention_decode(o, q, cache, tables, lens, lc.SCALE, 3000, workspace=ws)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    lens -= 1  # the graph reads the lengths of its replay
    graphs[0].replay()
    d = dict(c, lens=[2999, 9, 499], rows=[x[:-1] for x in c["rows"]])
    lc.check(outs[0], d)


def test_pairs_on_streams_in_graphs_and_beside_each_other():
    """Calls of more than 64 query rows: a captured one replayed with other lengths, two on two streams at once."""
    c = lc.make([900, 40, 333], 16, queries=[40, 9, 100])
    want = lc.run(c)
    cache, q = c["cache"].cuda(), c["q"].cuda()
    tables, lens = torch.from_numpy(c["tables"]).cuda(), torch.tensor(c["lens"], dtype=torch.int32).cuda()
    starts = torch.from_numpy(c["starts"]).cuda()
    outs = [torch.zeros_like(want) for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for o, st in zip(outs, streams):
            pkv.paged_latent_attention_multi_token(o, q, cache, tables, lens, starts, lc.SCALE, 100, 900, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs[:2])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.paged_latent_attention_multi_token(outs[2], q, cache, tables, lens, starts, lc.SCALE, 100, 900)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[2], want)
    lens -= 1
    g.replay()
    lc.check(outs[2], dict(c, lens=[x - 1 for x in c["lens"]], rows=[x[:-1] for x in c["rows"]]))


@pytest.mark.parametrize("dtype,NB", [(BF, 480000), (F32, 250000)])
@pytest.mark.parametrize("queries,H", [(None, 16), (None, 100), ([70, 3], 16)])
def test_a_pool_past_32_bits(dtype, NB, queries, H):
    """Blocks whose entries lie past 2^31 (float32) and 2^32 (bf16) entries of the pool: the results of a small pool, bit for bit."""
    c = lc.make([90, 130], H, dtype=dtype, queries=queries)
    want = lc.run(c)
    cache = torch.empty((NB, 16, 576), dtype=dtype, device="cuda")
    n = c["cache"].shape[0]
    cache[NB - n:] = c["cache"].cuda()
    cache[:n] = float("nan")  # where an offset cut to 32 bits might lead
    assert torch.equal(lc.run(dict(c, tables=c["tables"] + (NB - n)), cache=cache), want)
    # and rows written there
    src = c["rows"][1].cuda()
    f, at = pkv.rotary_frequencies(64, device="cuda"), torch.zeros(130, dtype=torch.int32, device="cuda")
    slots = torch.from_numpy(c["tables"][1].astype(np.int64)).cuda()[torch.arange(130, device="cuda") // 16] + (NB - n)
    slots = slots * 16 + torch.arange(130, device="cuda") % 16
    held = cache[NB - n:].clone()
    cache[NB - n:] = float("nan")
    pkv.latent_cache_write(src[:, :512], src[:, 512:], cache, slots, at, f)  # positions 0: rows as they are
    assert torch.equal(cache.view(-1, 576)[slots], src)
    assert torch.equal(held.view(-1, 576)[slots - (NB - n) * 16], src)


def test_an_output_16_bytes_off_a_sector():
    for queries in (None, [20, 9]):
        c = lc.make([300, 77], 16, queries=queries)
        want = lc.run(c)
        flat = torch.full((want.numel() + 24,), 7.0, dtype=BF, device="cuda")
        out = flat[8:8 + want.numel()].view(want.shape)
        assert torch.equal(lc.run(c, out=out), want)
        assert torch.all(flat[:8] == 7.0) and torch.all(flat[8 + want.numel():] == 7.0)


@pytest.mark.parametrize("V,H", [(512, 16), (256, 40)])
def test_write_and_attend_as_a_step(V, H):
    """Rows and queries rotated and stored by latent_cache_write, then attended: a prompt, a decode step, a verification."""
    B, L = 16, 75
    r = np.random.default_rng(4)
    f = pkv.rotary_frequencies(64)
    lat = torch.from_numpy(r.standard_normal((L, V)).astype(np.float32)).to(BF)
    key = torch.from_numpy(r.standard_normal((L, 64)).astype(np.float32)).to(BF)
    qn = torch.from_numpy(r.standard_normal((L, H, V + 64)).astype(np.float32)).to(BF)
    alloc = pkv.BlockAllocator(32, B)
    assert alloc.add_seq(0, 0) == 0
    slots = np.array([alloc.append_slot(0)[1] for _ in range(L)])
    tables = alloc.block_tables([0], cap=8)[0]
    cache = torch.full((32, B, V + 64), float("nan"), dtype=BF, device="cuda")
    dt, fd = torch.from_numpy(tables).cuda(), f.cuda()
    outs = []
    for a, b in ((0, 60), (60, 61), (61, 66), (66, L)):
        q = qn[a:b].cuda()
        pkv.latent_cache_write(lat[a:b].cuda(), key[a:b].cuda(), cache, torch.from_numpy(slots[a:b]).cuda(),
                               torch.arange(a, b, dtype=torch.int32, device="cuda"), fd, q_rope=q[..., V:], q_out=q[..., V:])
        out = torch.empty((b - a, H, V), dtype=BF, device="cuda")
        lens = torch.tensor([b], dtype=torch.int32, device="cuda")
        if b - a == 1:
            pkv.paged_latent_attention_decode(out, q, cache, dt, lens, lc.SCALE, 100)
        else:
            pkv.paged_latent_attention_multi_token(out, q, cache, dt, lens, torch.tensor([0, b - a], dtype=torch.int32, device="cuda"),
                                                   lc.SCALE, b - a, 100)
        outs.append(out)
    # the oracle on rows rounded to bf16 as stored
    turn = lambda x: torch.from_numpy(rotary.rotate(x.double().numpy(), np.arange(L), f.numpy())).to(BF)  # noqa: E731
    rows = torch.cat([lat, turn(key[:, None])[:, 0]], 1)
    q = torch.cat([qn[..., :V], turn(qn[..., V:])], 2)
    c = dict(rows=[rows], q=q, lens=[L], starts=np.array([0, L]), V=V, dtype=BF)
    want, tol = lc.expected(c)
    # a rotated entry may round to the neighbouring bf16 number: 64 of a score's products, each off by 2^-7 at most
    reach = np.abs(q[..., V:].double().numpy()) @ np.abs(rows[:, V:].double().numpy()).T
    tol = tol + 2 * 2 * 2.0 ** -7 * lc.SCALE * reach.max() / 64 * np.abs(rows[:, :V].double().numpy()).max()
    assert np.all(np.abs(torch.cat(outs).double().cpu().numpy() - want) <= tol)


def test_rotary_write_feeds_the_plain_attention():
    """kv_cache_write_rotary, then the decode and multi-token calls there were: the queries it wrote are read by them."""
    from oracle.multi_token import multi_token_attention
    T, Hq, Hkv, D, B = 50, 8, 2, 64, 16
    r = np.random.default_rng(8)
    qkv = torch.from_numpy(r.standard_normal((T, Hq + 2 * Hkv, D)).astype(np.float32)).to(BF)
    dev = qkv.cuda()
    f = pkv.rotary_frequencies(D)
    kc = torch.full((8, Hkv, B, D), float("nan"), dtype=BF, device="cuda")
    vc = torch.full_like(kc, float("nan"))
    q = torch.empty((T, Hq, D), dtype=BF, device="cuda")
    tables = torch.tensor([[5, 2, 7, 0]], dtype=torch.int32, device="cuda")
    at = torch.arange(T, device="cuda")
    slots = tables[0].long()[at // B] * B + at % B
    pkv.kv_cache_write_rotary(dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:], kc, vc, slots, at.int(), f.cuda(), q=dev[:, :Hq], q_out=q)
    out = torch.empty_like(q)
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    pkv.paged_attention_multi_token(out, q, kc, vc, tables, lens, torch.tensor([0, T], dtype=torch.int32, device="cuda"), 0.125, T, T)
    turn = lambda x: torch.from_numpy(rotary.rotate(x.double().numpy(), np.arange(T), f.numpy())).to(BF).double().numpy()  # noqa: E731
    qr, kr = turn(qkv[:, :Hq]), turn(qkv[:, Hq:Hq + Hkv])
    ref, = multi_token_attention([qr], [kr], [qkv[:, Hq + Hkv:].double().numpy()], 0.125)
    # weights and outputs rounded to bf16 (2^-8 each), rotated entries to a neighbouring number (scores off by 2^-7 of
    # products that are mostly far below 1): an order of magnitude under 0.1 for values of at most 4
    assert np.max(np.abs(out.double().cpu().numpy() - ref)) < 0.1
    one = torch.empty((1, Hq, D), dtype=BF, device="cuda")
    pkv.paged_attention_decode(one, q[-1:].contiguous(), kc, vc, tables, lens, 0.125, T)
    assert np.max(np.abs(one.double().cpu().numpy()[0] - ref[-1])) < 0.1


def test_refusals_on_the_device():
    c = lc.make([20], 4)
    q, cache = c["q"].cuda(), c["cache"].cuda()
    t, n = torch.from_numpy(c["tables"]).cuda(), torch.tensor([20], dtype=torch.int32).cuda()
    out = torch.empty((1, 4, 512), dtype=BF, device="cuda")
    for bad in (lambda: pkv.paged_latent_attention_decode(out.float(), q, cache, t, n, 1.0, 20),
                lambda: pkv.paged_latent_attention_decode(out, q, cache.float(), t, n, 1.0, 20),
                lambda: pkv.paged_latent_attention_decode(out, q, cache, t.long(), n, 1.0, 20),
                lambda: pkv.paged_latent_attention_decode(out, q, cache, t, n.long(), 1.0, 20),
                lambda: pkv.paged_latent_attention_decode(out.half(), q.half(), cache.half(), t, n, 1.0, 20)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(ValueError):
        pkv.paged_latent_attention_decode(out, q.transpose(1, 2).contiguous().transpose(1, 2), cache, t, n, 1.0, 20)
    with pytest.raises(pkv.PkvError):
        pkv.paged_latent_attention_decode(out, q, cache, t, n, 1.0, 20, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
