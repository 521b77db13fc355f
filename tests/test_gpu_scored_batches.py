"""Scored attention over large and unusual batches."""
import numpy as np
import pytest
import torch

import paged_kv_cache_279_gb300 as pkv
from harness import bits
from scored_cases import Case
from test_gpu_scored import run

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_errors():
    pkv.read_device_errors(clear=True)
    yield
    assert pkv.read_device_errors(clear=True) == 0


@pytest.mark.parametrize("opt", [dict(softcap=20.0), dict(alibi=True), dict(window=100, prefix=[3] * 27)],
                         ids=["cap", "alibi", "window"])
def test_many_long_prompts(opt):
    """More prompts of over 512 queries than one pass of the length scan takes (20 of four heads a KV head)."""
    r = np.random.default_rng(3)
    lens = [int(x) for x in r.integers(513, 700, 27)]
    lens[5], lens[20], lens[21], lens[26] = 0, 1, 700, 530
    qlens = [min(L, int(n)) for L, n in zip(lens, r.integers(1, 640, 27))]
    qlens[21], qlens[26] = 600, 530
    c = Case(lens, 4, 1, 64, 16, qlens=qlens, **opt)
    c.check(run(c, max_q_len=700))


@pytest.mark.parametrize("opt", [dict(softcap=20.0), dict(alibi=True, window=50)], ids=["cap", "alibi"])
def test_many_sequences_to_verify(opt):
    """More sequences than one pass of the length scan takes (640 of one query block each)."""
    r = np.random.default_rng(5)
    lens = [int(x) for x in r.integers(0, 200, 1500)]
    qlens = [min(L, int(n)) for L, n in zip(lens, r.integers(0, 6, 1500))]
    c = Case(lens, 2, 1, 64, 16, qlens=qlens, **opt)
    c.check(run(c))


def test_one_long_prompt_among_decodes():
    """A mixed step: the longest query count and length allowed for are those of one sequence only."""
    c = Case([900] + [40 + i for i in range(31)], 32, 8, 64, 16, qlens=[300] + [1] * 31, softcap=20.0)
    c.tables = np.concatenate([c.tables, np.full((32, 8192 - c.tables.shape[1]), -1, np.int32)], axis=1)
    c.check(run(c, max_seq_len=131072, max_q_len=131072))


def test_a_length_that_the_tables_do_not_hold():
    """max_seq_len beyond what the tables address changes nothing."""
    for kw in (dict(qlens=[5, 9, 1]), dict(), dict(rows=True)):
        c = Case([300, 77, 40], softcap=20.0, **kw)
        c.check(run(c, max_seq_len=2 ** 31 - 1))


@pytest.mark.parametrize("kind", ["bf16", "rows", "multi"])
def test_more_tiles_than_one_launch_counts(kind):
    """A batch whose longest possible contexts would pass 2^30 tiles is attended in parts.  The bound is that of the oracle's
    cases (scored_cases.Case.reference)."""
    S, H, D, B, maxB = (2100 if kind == "multi" else 300), 1024, 64, 16, 4096
    gen = torch.Generator(device="cuda").manual_seed(2)
    pools = {}
    for n in "kv":
        if kind == "rows":
            pools[n + "_cache"] = torch.randint(0, 120, (9, H, B, D), generator=gen, device="cuda", dtype=torch.uint8)
            pools[n + "_scales"] = torch.randint(122, 128, (9, H, B), generator=gen, device="cuda", dtype=torch.uint8)
        else:
            pools[n + "_cache"] = torch.randn((9, H, B, D), generator=gen, device="cuda").to(torch.bfloat16)
    q = torch.randn((S, H, D), generator=gen, device="cuda").to(torch.bfloat16)
    tables = torch.zeros((S, maxB), dtype=torch.int32, device="cuda")
    tables[:, :2] = torch.randint(0, 9, (S, 2), generator=gen, device="cuda", dtype=torch.int32)
    lens = torch.randint(1, 2 * B + 1, (S,), generator=gen, device="cuda", dtype=torch.int32)
    starts = torch.randint(0, 3, (S,), generator=gen, device="cuda", dtype=torch.int32)
    prefix = torch.randint(0, 9, (S,), generator=gen, device="cuda", dtype=torch.int32)

    out = torch.full_like(q, float("nan"))
    kw = dict(pools, block_tables=tables, seq_lens=lens, scale=0.1, max_seq_len=maxB * B, softcap=20.0, window=20,
              prefix_lens=prefix, key_starts=starts)
    if kind == "multi":
        pkv.paged_attention_multi_token_scored(out, q, **kw, max_q_len=1,
                                               q_starts=torch.arange(S + 1, dtype=torch.int32, device="cuda"))
    elif kind == "rows":
        pkv.paged_attention_decode_scored_fp8_rows(out, q, **kw)
    else:
        pkv.paged_attention_decode_scored(out, q, **kw)
    cache = {n: (pools[n + "_cache"].view(torch.float8_e4m3fn).double() *
                 torch.exp2(pools[n + "_scales"].double() - 127.0)[..., None]) if kind == "rows" else
             pools[n + "_cache"].double() for n in "kv"}
    # FP8 rows: an f16 weight w = p 2^ve is off by 2^-11 of itself or, as a subnormal, by 2^-25 where the largest one is 2^14,
    # that is by 2^-39 of p 2^ve <= 2^0 (scales here are at most 2^0); codes are at most 448, and 28 keys are seen at most
    floor = 28 * 448 * 2.0 ** -39 if kind == "rows" else 1e-30
    half, weight = torch.finfo(torch.bfloat16).eps / 2, 2.0 ** (-11 if kind == "rows" else -8)
    t = torch.arange(2 * B, device="cuda")
    for a in range(0, S, 100):
        k, v = (cache[n][tables[a:a + 100, :2].long()].transpose(1, 2).reshape(-1, H, 2 * B, D) for n in "kv")
        L, qa = lens[a:a + 100, None], q[a:a + 100].double()
        seen = (t < L) & (t >= starts[a:a + 100, None]) & ((t < prefix[a:a + 100, None]) | (L - 1 - t < 20))
        x = 20.0 * torch.tanh(0.1 * (qa[:, :, None] * k).sum(-1) / 20.0)
        w = torch.softmax(x.masked_fill(~seen[:, None], -float("inf")), -1)
        w = torch.where(seen.any(1)[:, None, None], w, torch.zeros_like(w))
        ref, size = ((w[..., None] * x).sum(2) for x in (v, v.abs()))
        top = 0.1 * (qa.abs()[:, :, None] * k.abs()).sum(-1).max()
        err = (D + 16) * 2.0 ** -24 * top + 2.0 ** -20 + 2.0 ** -18 * 20.0 + 2.0 ** -22 * top
        tol = 2 * (2 * err + weight + 2 * B * 2.0 ** -24) * size + half * ref.abs() * (1 + 2.0 ** -6) + floor
        worst = ((out[a:a + 100].double() - ref).abs() - tol).max().item()
        assert worst <= 0, (a, worst)


def test_parts_of_sequences_store_their_tokens_first():
    """New tokens of more sequences than one launch takes."""
    lens = [1 + (7 * i) % 23 for i in range(8300)]
    c = Case(lens, 2, 1, 64, 16, softcap=10.0)
    want, pools = c.pools(), c.pools()
    slot = torch.tensor([int(c.tables[s][(L - 1) // 16]) * 16 + (L - 1) % 16 for s, L in enumerate(lens)]).cuda()
    for n in ("k_cache", "v_cache"):
        pools[n][slot // 16, :, slot % 16] = float("nan")
    c.check(run(c, pools, k_new=torch.stack([k[-1] for k in c.ks]).cuda(), v_new=torch.stack([v[-1] for v in c.vs]).cuda()))
    for n in want:
        assert torch.equal(bits(pools[n]), bits(want[n]))


@pytest.mark.parametrize("kind", ["f32", "bf16", "rows"])
def test_the_workspace_of_a_type_suffices(kind):
    """Exactly the bytes that the size call gives for the query's type, none for one that needs none."""
    dt = torch.float32 if kind == "f32" else torch.bfloat16
    for lens, maxL in (([700, 33, 2000], 131072), ([100, 7], 500)):
        c = Case(lens, dtype=dt, rows=kind == "rows", softcap=20.0)
        need = pkv.paged_attention_decode_scored_workspace_size(len(lens), c.Hq, c.D, maxL, dt)
        ws = torch.randint(0, 256, (need + 256,), dtype=torch.uint8, device="cuda")
        after = ws[need:].clone()
        c.check(run(c, workspace=ws[:need] if need else None, max_seq_len=maxL))
        assert torch.equal(ws[need:], after)
        if need > 256:
            with pytest.raises(pkv.PkvError):
                run(c, workspace=ws[:need - 256], max_seq_len=maxL)


def test_many_queries_that_see_nothing():
    """Blocks of queries whose documents begin after them: zeros, beside queries that see their own."""
    c = Case([1000], 8, 2, 128, 16, qlens=[607], starts=[893] * 500 + [900] * 100 + [5000] * 7, softcap=20.0)
    got = run(c)
    c.check(got)
    assert torch.all(got[:507] == 0) and torch.all(got[600:] == 0) and torch.all(got[507:600].abs().sum(-1) > 0)
