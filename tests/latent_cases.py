"""Builds latent attention cases on the host, runs them on the GPU and holds the results against the oracle."""
import math

import numpy as np
import torch

import paged_kv_cache_279_gb300 as pkv
from oracle import latent as oracle_latent
from paged_kv_cache_279_gb300 import workloads as wl

SCALE = 1.0 / math.sqrt(192.0)


def make(lens, H, V=512, B=16, dtype=torch.bfloat16, queries=None, seed=0, fill=float("nan"), extra_blocks=2, size=1.0):
    """Contiguous rows a sequence and the paged pool that holds them, other slots ``fill``.  queries: tokens of each
    sequence (None: one each, a decode)."""
    D = V + 64
    r = np.random.default_rng(seed)
    draw = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32)).to(dtype)  # noqa: E731
    rows = [draw(L, D) for L in lens]
    nq = [1] * len(lens) if queries is None else list(queries)
    q = (draw(sum(nq), H, D).float() * size).to(dtype)
    counts = [-(-L // B) for L in lens]
    NB = sum(counts) + extra_blocks
    tables = wl.random_block_tables(counts, NB, max(1, max(counts)), seed + 1)
    cache = torch.full((NB, B, D), fill, dtype=dtype)
    for s, x in enumerate(rows):
        p = np.arange(x.shape[0])
        cache[torch.from_numpy(tables[s][p // B].astype(np.int64)), torch.from_numpy(p % B)] = x
    starts = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
    return dict(rows=rows, q=q, cache=cache, tables=tables, lens=list(lens), nq=nq, starts=starts, H=H, V=V, B=B, dtype=dtype,
                decode=queries is None)


def run(c, scale=SCALE, out=None, max_len=None, max_q=None, cache=None, **kw):
    T, H, _ = c["q"].shape
    if out is None:
        out = torch.full((T, H, c["V"]), 7.0, dtype=c["dtype"], device="cuda")
    cache = c["cache"].cuda() if cache is None else cache
    tables, lens = torch.from_numpy(np.ascontiguousarray(c["tables"])).cuda(), torch.tensor(c["lens"], dtype=torch.int32).cuda()
    max_len = max_len or max(1, max(c["lens"]))
    if c["decode"]:
        pkv.paged_latent_attention_decode(out, c["q"].cuda(), cache, tables, lens, scale, max_len, **kw)
    else:
        pkv.paged_latent_attention_multi_token(out, c["q"].cuda(), cache, tables, lens, torch.from_numpy(c["starts"]).cuda(), scale,
                                               max_q or max(1, max(c["nq"])), max_len, **kw)
    torch.cuda.synchronize()
    return out


def expected(c, scale=SCALE):
    """(out, tolerance) of every query row.  Rounding errors, with u = 2^-24: a score, a sum of D products in float32, is
    off by at most reach (D + 4) u (reach: the sum of the products' sizes), its weight's exponential by that and 2^-21
    (two approximations and the reference they are taken against), the sums over a context of L tokens by (L + 2) u of
    their sizes.  bf16: a weight is rounded once, by 2^-8 of itself, and numerator and denominator hold the same
    rounded weights or differ by that; the output once more."""
    q = c["q"].double().numpy()
    parts = [q[c["starts"][s]:c["starts"][s + 1]] for s in range(len(c["lens"]))]
    res = oracle_latent.latent_attention(parts, [x.double().numpy() for x in c["rows"]], scale, c["V"])
    out, spread, reach = (np.concatenate([r[k] for r in res]) for k in range(3))
    u = 2.0 ** -24
    D, L = c["V"] + 64, max(c["lens"])
    rel = 2 * (reach * (D + 4) * u + 2.0 ** -21 + (L + 2) * u)
    half = torch.finfo(c["dtype"]).eps / 2
    if c["dtype"] == torch.bfloat16:
        rel = rel + 2 * half
    return out, rel * spread + half * np.abs(out) + 1e-37


def check(got, c, scale=SCALE, what=""):
    want, tol = expected(c, scale)
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= tol), f"{what}: {np.max(err / tol):.3g} of the tolerance, {np.sum(~(err <= tol))} of {err.size} outside"
