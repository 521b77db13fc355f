"""GPU: latent attention with lengths, blocks and query starts that are out of range, and short contexts cut into shares, on
every kernel: float32, up to 64 bf16 query rows a sequence, more than 64."""
import numpy as np
import pytest
import torch

import latent_cases as lc
import latent_more as lm
import paged_kv_cache_279_gb300 as pkv

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
KERNELS = [(F32, 3, None), (F32, 3, [5, 3]), (BF, 16, None), (BF, 40, None), (BF, 128, None), (BF, 4, [5, 3]), (BF, 16, [4, 4]), (BF, 16, [40, 9]),
           (BF, 2, [90, 60])]


@pytest.fixture(autouse=True)
def _clear_errors():
    pkv.read_device_errors(clear=True)
    yield
    assert pkv.read_device_errors(clear=True) == 0


@pytest.mark.parametrize("dtype,H,queries", KERNELS)
@pytest.mark.parametrize("L,max_len", [(112, 5000), (112, 112), (3008, 10 ** 6), (3000, 3000)])
def test_lengths_above_the_limit_are_cut(dtype, H, queries, L, max_len):
    """By the block table (all of its tokens are finite rows), or by max_seq_len."""
    c = lc.make([L, 64], H, 512, 16, dtype, queries)
    c["tables"][1, 4:] = -1
    for claim in (L + 1, 2 ** 31 - 1):
        got = lc.run(dict(c, lens=[claim, 64]), max_len=max_len)
        assert pkv.read_device_errors(clear=True) == pkv.DEVERR_SEQ_LEN
        lc.check(got, c)


@pytest.mark.parametrize("dtype,H,queries", KERNELS)
@pytest.mark.parametrize("table", [0, 8192])
def test_negative_lengths_are_empty_contexts(dtype, H, queries, table):
    c = lc.make([112, 64], H, 512, 16, dtype, queries)
    c = lm.wide(c, table) if table else c
    for claim in (-1, -2 ** 31):
        got = lc.run(dict(c, lens=[claim, 64]), max_len=10 ** 6)
        assert pkv.read_device_errors(clear=True) == pkv.DEVERR_SEQ_LEN
        n = c["nq"][0]
        assert torch.all(got[:n] == 0)
        want, tol = lc.expected(c)
        lm.check(got[n:], (want[n:], tol[n:]))


@pytest.mark.parametrize("dtype,H,queries", KERNELS)
@pytest.mark.parametrize("table", [0, 8192])
def test_blocks_out_of_range_are_left_out(dtype, H, queries, table):
    c = lc.make([150, 64], H, 512, 16, dtype, queries)
    c = lm.wide(c, table) if table else c
    for bad, which in ((-1, [2]), (c["cache"].shape[0], [9]), (2 ** 31 - 1, [0, 3, 4, 8]), (-2 ** 31, range(10))):
        t, dead = c["tables"].copy(), lm.none_dead(c)
        for b in which:
            t[0, b] = bad
            dead[0][:, 16 * b:16 * b + 16] = True
        got = lc.run(dict(c, tables=t), max_len=10 ** 6)
        assert pkv.read_device_errors(clear=True) == pkv.DEVERR_BLOCK_ID
        lm.check(got, lm.expected(c, dead))


@pytest.mark.parametrize("dtype,H,n", [(F32, 3, 4), (BF, 16, 4), (BF, 4, 4), (BF, 16, 40), (BF, 100, 5)])
@pytest.mark.parametrize("table", [0, 8192])
def test_query_starts_out_of_range(dtype, H, n, table):
    c = lc.make([100, 64, 50], H, 512, 16, dtype, queries=[n] * 3)
    c = lm.wide(c, table) if table else c
    want, tol = lc.expected(c)
    for starts in ([0, n, 100 * n, 3 * n], [0, n, -1, 3 * n], [0, n, 2 * n, 3 * n + 1], [0, n, 2 * n, 2 ** 31 - 1]):
        got = lc.run(dict(c, starts=np.array(starts, dtype=np.int32)), max_len=10 ** 6, max_q=n)
        assert pkv.read_device_errors(clear=True) & pkv.DEVERR_SEQ_LEN
        k = n if starts[2] != 2 * n else 2 * n
        lm.check(got[:k], (want[:k], tol[:k]))
    got = lc.run(c, max_len=10 ** 6, max_q=n - 1)  # queries past max_q are not attended, and their rows left as they were
    assert pkv.read_device_errors(clear=True) == pkv.DEVERR_SEQ_LEN
    keep = torch.arange(3 * n) % n != n - 1
    assert torch.all(got[~keep.cuda()] == 7.0)
    lm.check(got[keep.cuda()], (want[keep.numpy()], tol[keep.numpy()]))


@pytest.mark.parametrize("lens,H,V,B", [([1, 17, 33, 100], 4, 512, 16), ([1], 1, 256, 8), ([64], 16, 512, 64), ([65, 63, 128], 3, 256, 32),
                                        ([0, 129, 0, 1, 700], 33, 512, 16), ([40] * 9, 65, 256, 16), ([300, 2, 0], 128, 512, 8), ([129, 128, 127], 100, 512, 64),
                                        ([48, 96, 49, 47], 20, 512, 16), ([130] * 170, 10, 256, 8), ([5, 0, 3] * 70, 70, 512, 32)])
def test_short_contexts_cut(lens, H, V, B):
    c = lm.wide(lc.make(lens, H, V, B))
    lc.check(lc.run(c, max_len=10 ** 6), c)


@pytest.mark.parametrize("lens,nq,H,V,B", [([7], [7], 4, 512, 16), ([100, 33, 1], [5, 1, 1], 4, 512, 16), ([200], [130], 3, 256, 8),
                                           ([64, 65], [64, 65], 1, 512, 64), ([300, 40], [9, 40], 33, 256, 32), ([90, 500], [64, 3], 128, 512, 16),
                                           ([20, 30, 40], [0, 5, 0], 16, 512, 16), ([33] * 120, [1, 2, 0, 4] * 30, 16, 512, 16),
                                           ([260, 0, 129], [70, 0, 129], 7, 512, 16), ([130, 1, 2] * 30, [9, 1, 2] * 30, 8, 256, 8)])
def test_short_contexts_of_several_queries_cut(lens, nq, H, V, B):
    c = lm.wide(lc.make(lens, H, V, B, queries=nq))
    lc.check(lc.run(c, max_len=10 ** 6), c)


@pytest.mark.parametrize("queries,H", [(None, 16), (None, 100), ([5, 3], 6), ([50, 70], 6)])
def test_what_is_not_seen_does_not_matter_to_cut_contexts(queries, H):
    want = lc.run(lm.wide(lc.make([77, 130], H, 512, 16, BF, queries, fill=0.0)), max_len=10 ** 6)
    for fill in (float("nan"), float("inf"), -float("inf"), torch.finfo(BF).max, torch.finfo(BF).min):
        d = lm.wide(lc.make([77, 130], H, 512, 16, BF, queries, fill=fill))
        assert torch.equal(lc.run(d, max_len=10 ** 6), want)


@pytest.mark.parametrize("L,more,H", [(3, 2, 4), (3, 40, 4), (60, 70, 16), (700, 100, 5), (0, 50, 16), (0, 3, 2)])
def test_more_queries_than_tokens_cut(L, more, H):
    c = lc.make([L, 40], H, queries=[L, 4])
    r = torch.from_numpy(np.random.default_rng(8).standard_normal((more, H, 576)).astype(np.float32)).to(BF)
    c["q"] = torch.cat([r, c["q"]])
    c["starts"] = np.array([0, L + more, L + more + 4], dtype=np.int32)
    c["nq"] = [L + more, 4]
    out = lc.run(lm.wide(c), max_len=10 ** 6)
    assert pkv.read_device_errors(clear=True) == pkv.DEVERR_SEQ_LEN
    assert torch.all(out[:more] == 0)
    lc.check(out, c)


@pytest.mark.parametrize("queries,H", [(None, 16), (None, 128), ([5, 3, 2], 8), ([50, 70, 1], 6)])
def test_cut_calls_repeat_themselves_in_graphs_too(queries, H):
    """A captured call replayed with other lengths; two graphs that share a workspace; the same bits every time."""
    c = lm.wide(lc.make([400, 77, 30], H, 512, 16, BF, queries))
    want = lc.run(c, max_len=8192)
    cache, q = c["cache"].cuda(), c["q"].cuda()
    tables, lens = torch.from_numpy(c["tables"]).cuda(), torch.tensor(c["lens"], dtype=torch.int32).cuda()
    starts = torch.from_numpy(c["starts"]).cuda()
    n = pkv.paged_latent_attention_workspace_size(q.shape[0], H, 512, 8192)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")

    def call(o):
        if queries is None:
            pkv.paged_latent_attention_decode(o, q, cache, tables, lens, lc.SCALE, 8192, workspace=ws)
        else:
            pkv.paged_latent_attention_multi_token(o, q, cache, tables, lens, starts, lc.SCALE, max(queries), 8192, workspace=ws)
    outs, graphs = [torch.zeros_like(want) for _ in range(2)], []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(o)
        graphs.append(g)
    for _ in range(4):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    lens -= 1
    graphs[1].replay()
    lc.check(outs[1], dict(c, lens=[x - 1 for x in c["lens"]], rows=[x[:-1] for x in c["rows"]]))


@pytest.mark.parametrize("dtype,H,n", [(F32, 3, 4), (BF, 16, 4), (BF, 16, 40), (BF, 100, 5)])
@pytest.mark.parametrize("table", [0, 8192])
def test_a_batch_without_queries(dtype, H, n, table):
    """No sequence owns a row: nothing is written; empty sequences around one that does, and empty contexts among them."""
    c = lc.make([100, 64, 50], H, 512, 16, dtype, queries=[0, n, 0])
    c = lm.wide(c, table) if table else c
    got = lc.run(dict(c, starts=np.zeros(4, dtype=np.int32)), max_len=10 ** 6)
    assert torch.all(got == 7.0)
    got = lc.run(dict(c, lens=[0, 64, 0]), max_len=10 ** 6)
    lc.check(got, c)
