"""Cases of the scored attention and row-scaled FP8 cache operators, for timing and checking them.

Five operators of a paged KV cache:

* write: kv_cache_write_fp8_rows -- new K/V rows quantised to E4M3 as they are stored, one power-of-two scale for
  each row (token, KV head);
* read: kv_cache_read_fp8_rows -- the values of such rows, gathered back by slot;
* decode: paged_attention_decode_scored -- one query a sequence over a float32 or bfloat16 cache, its scores capped
  by a tanh and / or biased by distance, its keys limited by a window, a document start and an always visible prefix;
* rows: paged_attention_decode_scored_fp8_rows -- the same over the row-scaled FP8 cache;
* multi: paged_attention_multi_token_scored -- the same for several causal queries a sequence.

Scores, for the query at position p of a context of L tokens and the key at t < L, with x = scale * q.k:
    x <- softcap * tanh(x / softcap)          (softcap > 0)
    x <- x - slope[head] * |p - t|            (slopes given)
and the key is seen if t >= key_start and (t < prefix_len, or t <= p and, with a window, p - t < window).  A query that
sees nothing gets zeros.

With ``own`` false, run() computes the plain forms in elementary torch operations; with ``own`` true it makes the
calls of the framework.
"""
import math
import random

import numpy as np
import torch

own = False
DEV = "cuda"


# ---------------------------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------------------------
def _write(name, **k):
    return dict({"op": "write", "tokens": 64, "kv_heads": 8, "head_dim": 128, "block": 16, "dtype": "bf16"}, **k, name=name)


def _attend(name, op, **k):
    c = {"op": op, "seqs": 64, "len_lo": 64, "len_hi": 2048, "heads": 32, "kv_heads": 8, "head_dim": 128, "block": 16,
         "dtype": "bf16", "softcap": 0.0, "alibi": False, "window": 0, "prefix": 0, "docs": 0, "append": False}
    if op == "multi":
        c["queries"] = 5
    return dict(c, **k, name=name)


def listed():
    return [
        # one decode step's new tokens of 64 sequences: latency
        _write("write 64 tokens"),
        # the prompts of a prefill batch
        _write("write 16384 tokens", tokens=16384),
        # one stored prompt brought back, its length no multiple of anything
        _write("read 1001 tokens", op="read", tokens=1001),
        # the contexts of a batch brought back into plain rows
        _write("read 65536 tokens", op="read", tokens=65536),
        # four short sequences in float32: the smallest call
        _attend("decode tiny float32 cap alibi", "decode", seqs=4, len_lo=1, len_hi=100, heads=4, kv_heads=4, head_dim=64,
                dtype="f32", softcap=30.0, alibi=True),
        # the serving step: 64 sequences of mixed lengths, capped scores, the new token stored in the same call
        _attend("decode 64 x 64..2048 cap append", "decode", softcap=30.0, append=True),
        # long contexts read through a window, the first tokens always visible
        _attend("decode 8 x 16000 window", "decode", seqs=8, len_lo=16000, len_hi=16000, window=4096, prefix=4),
        # the serving step over the quantised cache
        _attend("rows 64 x 64..2048 cap", "rows", softcap=30.0),
        # long contexts over the quantised cache, biased by distance
        _attend("rows 8 x 16000 alibi", "rows", seqs=8, len_lo=16000, len_hi=16000, alibi=True),
        # five drafted tokens a sequence to verify
        _attend("multi 64 x 5 cap", "multi", softcap=30.0),
        # a prefill chunk at the end of 4096 tokens
        _attend("multi 8 x 512 of 4096 cap", "multi", seqs=8, len_lo=4096, len_hi=4096, queries=512, softcap=30.0),
        # whole prompts packed from several documents, biased by distance
        _attend("multi 4 prompts of documents alibi", "multi", seqs=4, len_lo=3200, len_hi=4000, queries=4000, docs=8,
                alibi=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "decode", "decode", "rows", "rows", "multi", "multi", "multi"])
    if op in ("write", "read"):
        heads = rng.choice([1, 2, 3, 4, 8])
        return {"op": op, "tokens": max(1, min(_log(rng, 1, 40000), 65536 * 8 // heads)), "kv_heads": heads,
                "head_dim": rng.choice([64, 128]), "block": rng.choice([16, 32]), "dtype": rng.choice(["bf16", "bf16", "f32"])}
    kv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    c = {"op": op, "kv_heads": kv, "heads": kv * group, "head_dim": rng.choice([64, 128]),
         "block": rng.choice([16, 32] if op == "rows" else [8, 16, 32]),
         "dtype": rng.choice(["bf16", "bf16", "bf16", "f32"]) if op == "decode" else "bf16"}
    c["seqs"] = _log(rng, 1, 64)
    top = min(16000, (32768 if c["dtype"] == "f32" else 65536) // c["seqs"])
    c["len_hi"] = _log(rng, 1, top)
    c["len_lo"] = max(1, _log(rng, max(1, c["len_hi"] // 30), c["len_hi"]))
    c["softcap"] = rng.choice([0.0, 15.0, 30.0, 50.0])
    c["alibi"] = rng.random() < 0.4
    c["window"] = rng.choice([0, 0, _log(rng, 1, 4096)])
    c["prefix"] = rng.choice([0, 0, _log(rng, 1, max(1, c["len_hi"] // 2))])
    c["docs"] = rng.choice([0, 0, 0, rng.randint(2, 9)])
    c["append"] = op == "decode" and rng.random() < 0.3
    if op == "multi":
        most = max(1, 2 ** 27 // (c["seqs"] * c["len_hi"] * c["heads"]))
        c["queries"] = _log(rng, 1, min(most, c["len_hi"], 2048))
    return c


def _plan(case, seed):
    """Lengths, query counts, document starts and prefixes of a case, on the host.  The lengths are the case's own, their
    order the seed's: every seed's batch holds as many tokens and blocks."""
    S = case["seqs"]
    r = random.Random("%d to %d" % (case["len_lo"], case["len_hi"]))
    lens = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(S)]
    r = random.Random("%d plan" % seed)
    r.shuffle(lens)
    nq = [min(case.get("queries", 1), L) for L in lens]
    prefix = [min(case["prefix"], L) for L in lens] if case["prefix"] else None
    starts = None
    if case["docs"]:  # each sequence's context is a row of documents; a query's keys begin with its own
        starts = []
        for L, n in zip(lens, nq):
            cuts = np.array([0] + sorted(r.randint(0, L) for _ in range(case["docs"] - 1)), dtype=np.int64)
            p = np.arange(L - n, L, dtype=np.int64)
            starts.append(cuts[np.searchsorted(cuts, p, side="right") - 1])
    return lens, nq, prefix, starts


def work(case):
    D, Hkv = case["head_dim"], case["kv_heads"]
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] in ("write", "read"):
        T = case["tokens"]
        return {"bytes": T * (2 * Hkv * D * size + 2 * Hkv * (D + 1) + 8), "flops": T * 2 * Hkv * D * 2}
    lens, nq, prefix, starts = _plan(case, 0)
    Hq = case["heads"]
    keys, pairs = 0, 0
    for s, (L, n) in enumerate(zip(lens, nq)):
        p = np.arange(L - n, L, dtype=np.int64)
        ks = starts[s] if starts is not None else np.zeros(n, dtype=np.int64)
        lo = np.maximum(ks, p - case["window"] + 1) if case["window"] else ks
        hi = p + 1
        pre = np.minimum(prefix[s], L) if prefix else 0
        pairs += int((hi - lo).sum() + np.maximum(0, np.minimum(pre, lo) - ks).sum() + np.maximum(0, pre - np.maximum(hi, ks)).sum())
        seen = np.zeros(L + 1, dtype=np.int64)
        np.add.at(seen, lo, 1)
        np.add.at(seen, hi, -1)
        if prefix:
            np.add.at(seen, np.minimum(ks, pre), 1)
            np.add.at(seen, np.full(n, pre), -1)
        keys += int((np.cumsum(seen)[:L] > 0).sum())
    kv = 2 * Hkv * (D + 1) if case["op"] == "rows" else 2 * Hkv * D * size
    return {"bytes": keys * kv + sum(nq) * 2 * Hq * D * size, "flops": 4 * D * Hq * pairs}


# ---------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------
def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _rows(shape, gen, dtype):
    """Rows of a K or V cache: N(0, 1) entries, each row's size spread around 1, a few channels larger than the rest."""
    x = torch.randn(shape, generator=gen, device=DEV)
    x *= torch.exp(0.5 * torch.randn(shape[:-1] + (1,), generator=gen, device=DEV))
    x[..., 5] *= 4.0
    return x.to(dtype)


def _quantise(x):
    """(codes, exponent bytes) of rows x[..., D]: the smallest power of two 2^e with max |x| <= 448 * 2^e, e + 127 held
    in 27 .. 247; code = the nearest E4M3 value of x / 2^e."""
    x = x.float()
    _, e = torch.frexp(x.abs().amax(-1, keepdim=True) / 448.0)
    # frexp: a = f * 2^e with f in [0.5, 1); a power of two itself needs no larger one
    e = torch.where(x.abs().amax(-1, keepdim=True) <= torch.ldexp(torch.full_like(x[..., :1], 448.0), e - 1), e - 1, e)
    e = e.clamp(-100, 120)
    codes = torch.ldexp(x, -e).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8).squeeze(-1)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    D, Hkv, B = case["head_dim"], case["kv_heads"], case["block"]
    dt = _dtype(case)
    st = {"case": case, "dtype": dt}
    if case["op"] in ("write", "read"):
        T = case["tokens"]
        used = -(-T // B)
        NB = used + used // 10 + 1
        # consecutive positions of contexts whose blocks lie anywhere in the pool
        blocks = torch.randperm(NB, generator=gen, device=DEV)[:used]
        pos = torch.arange(T, device=DEV)
        st["slots"] = blocks[pos // B] * B + pos % B
        if case["op"] == "write":
            st["k_new"], st["v_new"] = _rows((T, Hkv, D), gen, dt), _rows((T, Hkv, D), gen, dt)
            st["kc"] = torch.zeros((NB, Hkv, B, D), dtype=torch.uint8, device=DEV)
            st["vc"] = torch.zeros_like(st["kc"])
            st["ks"] = torch.zeros((NB, Hkv, B), dtype=torch.uint8, device=DEV)
            st["vs"] = torch.zeros_like(st["ks"])
        else:
            for n in "kv":
                c, e = _quantise(_rows((NB, Hkv, B, D), gen, torch.bfloat16))
                st[n + "c"], st[n + "s"] = c.view(torch.uint8), e
        return st
    lens, nq, prefix, starts = _plan(case, seed)
    S, Hq, T = case["seqs"], case["heads"], sum(nq)
    counts = [-(-L // B) for L in lens]
    maxb, need = max(counts), sum(counts)
    NB = need + need // 10 + 1
    ids = torch.randperm(NB, generator=gen, device=DEV).to(torch.int32).cpu().numpy()
    tables = np.zeros((S, maxb), dtype=np.int32)
    at = 0
    for s, n in enumerate(counts):
        tables[s, :n] = ids[at:at + n]
        at += n
    q_starts = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
    st["tables"], st["lens"] = torch.from_numpy(tables).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    st["q_starts"] = torch.from_numpy(q_starts).to(DEV)
    st["max_q"], st["max_len"] = max(nq), max(lens)
    st["prefix"] = torch.tensor(prefix, dtype=torch.int32, device=DEV) if prefix else None
    st["starts"] = torch.from_numpy(np.concatenate(starts).astype(np.int32)).to(DEV) if starts is not None else None
    st["slopes"] = torch.exp2(-8.0 * torch.arange(1, Hq + 1, device=DEV) / Hq).float() if case["alibi"] else None
    st["scale"] = 1.0 / math.sqrt(D)
    st["q"] = (3.0 * torch.randn((T, Hq, D), generator=gen, device=DEV)).to(dt)
    st["append"] = None
    if case["op"] == "rows":
        for n in "kv":
            c, e = _quantise(_rows((NB, Hkv, B, D), gen, torch.bfloat16))
            st[n + "c"], st[n + "s"] = c.view(torch.uint8), e
    else:
        st["kc"] = torch.randn((NB, Hkv, B, D), generator=gen, device=DEV).to(dt)
        st["vc"] = torch.randn((NB, Hkv, B, D), generator=gen, device=DEV).to(dt)
        if case["append"]:
            st["append"] = tuple(torch.randn((S, Hkv, D), generator=gen, device=DEV).to(dt) for _ in "kv")
    return st


# ---------------------------------------------------------------------------------------------------------------
# The operators
# ---------------------------------------------------------------------------------------------------------------
def run(st):
    op = st["case"]["op"]
    if own:
        return {"write": _own_write, "read": _own_read, "decode": _own_decode, "rows": _own_rows, "multi": _own_multi}[op](st)
    return {"write": _plain_write, "read": _plain_read, "decode": _plain_decode, "rows": _plain_rows, "multi": _plain_multi}[op](st)


def _codes(st):
    return {"k": st["kc"].view(torch.float8_e4m3fn), "v": st["vc"].view(torch.float8_e4m3fn), "ks": st["ks"], "vs": st["vs"]}


def _own_write(st):
    import paged_kv_cache_279_gb300 as pkv
    pkv.kv_cache_write_fp8_rows(st["k_new"], st["v_new"], st["kc"], st["vc"], st["ks"], st["vs"], st["slots"])
    return _codes(st)


def _plain_write(st):
    B = st["case"]["block"]
    blk, off = st["slots"] // B, st["slots"] % B
    kc, ks = _quantise(st["k_new"])
    vc, vs = _quantise(st["v_new"])
    st["kc"][blk, :, off], st["ks"][blk, :, off] = kc.view(torch.uint8), ks
    st["vc"][blk, :, off], st["vs"][blk, :, off] = vc.view(torch.uint8), vs
    return _codes(st)


def _own_read(st):
    import paged_kv_cache_279_gb300 as pkv
    c = st["case"]
    k = torch.empty((c["tokens"], c["kv_heads"], c["head_dim"]), dtype=st["dtype"], device=DEV)
    v = torch.empty_like(k)
    pkv.kv_cache_read_fp8_rows(k, v, st["kc"], st["vc"], st["ks"], st["vs"], st["slots"])
    return k, v


def _values(codes, exps):
    return torch.ldexp(codes.view(torch.float8_e4m3fn).float(), exps.to(torch.int32).unsqueeze(-1) - 127)


def _plain_read(st):
    B = st["case"]["block"]
    blk, off = st["slots"] // B, st["slots"] % B
    return (_values(st["kc"][blk, :, off], st["ks"][blk, :, off]).to(st["dtype"]),
            _values(st["vc"][blk, :, off], st["vs"][blk, :, off]).to(st["dtype"]))


def _score_args(st):
    return {"softcap": st["case"]["softcap"], "alibi_slopes": st["slopes"], "window": st["case"]["window"],
            "prefix_lens": st["prefix"], "key_starts": st["starts"]}


def _own_decode(st):
    import paged_kv_cache_279_gb300 as pkv
    out = torch.empty_like(st["q"])
    k_new, v_new = st["append"] or (None, None)
    pkv.paged_attention_decode_scored(out, st["q"], st["kc"], st["vc"], st["tables"], st["lens"], st["scale"], st["max_len"],
                                      k_new=k_new, v_new=v_new, **_score_args(st))
    return (out, st["kc"], st["vc"]) if st["append"] else out


def _own_rows(st):
    import paged_kv_cache_279_gb300 as pkv
    out = torch.empty_like(st["q"])
    pkv.paged_attention_decode_scored_fp8_rows(out, st["q"], st["kc"], st["vc"], st["ks"], st["vs"], st["tables"], st["lens"],
                                               st["scale"], st["max_len"], **_score_args(st))
    return out


def _own_multi(st):
    import paged_kv_cache_279_gb300 as pkv
    out = torch.empty_like(st["q"])
    pkv.paged_attention_multi_token_scored(out, st["q"], st["kc"], st["vc"], st["tables"], st["lens"], st["q_starts"],
                                           st["scale"], st["max_q"], st["max_len"], **_score_args(st))
    return out


def _plain_attend(st, k, v):
    """Attention of the packed queries over contexts k, v [S, L, Hkv, D], in float32: the whole matrix of scores, masked."""
    c = st["case"]
    S, L, Hkv, D = k.shape
    G, Q = c["heads"] // Hkv, st["max_q"]
    lens, q0 = st["lens"].long(), st["q_starts"].long()
    nq = q0[1:] - q0[:-1]
    i = torch.arange(Q, device=DEV)
    live = i < nq[:, None]                                              # [S, Q]
    row = torch.where(live, q0[:-1, None] + i, 0)
    q = st["q"][row].float().reshape(S, Q, Hkv, G, D)
    x = torch.einsum("sqhgd,slhd->shgql", q, k) * st["scale"]
    if c["softcap"]:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    t = torch.arange(L, device=DEV)
    p = (lens - nq)[:, None] + i                                        # positions [S, Q]
    away = p[:, :, None] - t
    if st["slopes"] is not None:
        x = x - st["slopes"].reshape(1, Hkv, G, 1, 1) * away.abs()[:, None, None].float()
    seen = away >= 0
    if c["window"]:
        seen = seen & (away < c["window"])
    if st["prefix"] is not None:
        seen = seen | (t < st["prefix"].long()[:, None, None])
    if st["starts"] is not None:
        seen = seen & (t >= st["starts"].long()[row][:, :, None])
    seen = seen & (t < lens[:, None, None])
    x = x.masked_fill(~seen[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    w = torch.exp(x - torch.where(top == float("-inf"), 0.0, top))
    total = w.sum(-1, keepdim=True)
    o = torch.einsum("shgql,slhd->sqhgd", w / torch.where(total == 0, 1.0, total), v)
    return o.reshape(S, Q, Hkv * G, D)[live].to(st["q"].dtype)


def _contexts(st, pool):
    """A pool [NB, Hkv, B, ...] as contexts [S, L, Hkv, ...] through the block tables; zeros past a context's end."""
    B = st["case"]["block"]
    x = pool[st["tables"].long()].transpose(2, 3).flatten(1, 2)[:, :st["max_len"]]
    dead = torch.arange(x.shape[1], device=DEV) >= st["lens"].long()[:, None]
    return x.masked_fill(dead.reshape(dead.shape + (1,) * (x.dim() - 2)), 0)


def _plain_decode(st):
    if st["append"]:
        B = st["case"]["block"]
        p = st["lens"].long() - 1
        blk = st["tables"].long().gather(1, (p // B)[:, None])[:, 0]
        st["kc"][blk, :, p % B], st["vc"][blk, :, p % B] = st["append"]
    o = _plain_attend(st, _contexts(st, st["kc"]).float(), _contexts(st, st["vc"]).float())
    return (o, st["kc"], st["vc"]) if st["append"] else o


def _plain_rows(st):
    return _plain_attend(st, _values(_contexts(st, st["kc"]), _contexts(st, st["ks"])),
                         _values(_contexts(st, st["vc"]), _contexts(st, st["vs"])))


def _plain_multi(st):
    return _plain_attend(st, _contexts(st, st["kc"]).float(), _contexts(st, st["vc"]).float())


# ---------------------------------------------------------------------------------------------------------------
# The definition, in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def _exact_rows(x):
    """Row-scaled E4M3 of x[..., D]: (values of the codes, exponent bytes), from the format's definition."""
    x = x.double()
    a = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(a > 0, a, 1.0) / 448.0))
    e = torch.where(a > 448.0 * torch.exp2(e), e + 1, e)                # log2 may round either way at a border
    e = torch.where(a <= 448.0 * torch.exp2(e - 1), e - 1, e)
    e = torch.where(a > 0, e, -100.0).clamp(-100, 120)
    y = x * torch.exp2(-e)
    step = torch.exp2(torch.floor(torch.log2(torch.where(y == 0, 1.0, y.abs()))).clamp(min=-6) - 3)  # 3 fraction bits, subnormals below 2^-6
    return (torch.round(y / step) * step).clamp(-448, 448), (e + 127).to(torch.uint8).squeeze(-1)


def exact(case, seed):
    st = prepare(case, seed)
    B, D, Hkv = case["block"], case["head_dim"], case["kv_heads"]
    if case["op"] == "write":
        got = {}
        for n in "kv":
            c, e = _exact_rows(st[n + "_new"])
            blk, off = torch.div(st["slots"], B, rounding_mode="floor"), st["slots"] % B
            got[n] = torch.zeros(st[n + "c"].shape, dtype=torch.float64, device=DEV)
            got[n][blk, :, off] = c
            got[n + "s"] = torch.zeros_like(st[n + "s"])
            got[n + "s"][blk, :, off] = e
        return got
    value = lambda codes, exps: codes.view(torch.float8_e4m3fn).double() * torch.exp2(exps.double() - 127).unsqueeze(-1)  # noqa: E731
    if case["op"] == "read":
        at = torch.stack([torch.div(st["slots"], B, rounding_mode="floor"), st["slots"] % B], 1)
        return tuple(value(st[n + "c"], st[n + "s"])[at[:, 0], :, at[:, 1]] for n in "kv")
    Hq, outs = case["heads"], []
    q0 = st["q_starts"].tolist()
    for s, L in enumerate(st["lens"].tolist()):  # each sequence by itself, its context laid out in order
        ids = st["tables"][s, :-(-L // B)].long()
        if case["op"] == "rows":
            k, v = (value(st[n + "c"][ids], st[n + "s"][ids]) for n in "kv")
        else:
            k, v = (st[n + "c"][ids].double() for n in "kv")
        k, v = (x.permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :L].clone() for x in (k, v))
        if st["append"]:
            k[:, L - 1], v[:, L - 1] = (x[s].double() for x in st["append"])
        q = st["q"][q0[s]:q0[s + 1]].double()
        n = q.shape[0]
        pos = torch.arange(L - n, L, device=DEV, dtype=torch.float64)[:, None]
        t = torch.arange(L, device=DEV, dtype=torch.float64)[None]
        hidden = t > pos
        if case["window"]:
            hidden |= pos - t >= case["window"]
        if st["prefix"] is not None:
            hidden &= t >= float(st["prefix"][s])
        if st["starts"] is not None:
            hidden |= t < st["starts"][q0[s]:q0[s + 1], None].double()
        o = torch.empty((n, Hq, D), dtype=torch.float64, device=DEV)
        for h in range(Hq):
            g = h // (Hq // Hkv)
            x = q[:, h] @ k[g].T * st["scale"]
            if case["softcap"]:
                x = torch.tanh(x / case["softcap"]) * case["softcap"]
            if st["slopes"] is not None:
                x -= st["slopes"][h].double() * (pos - t).abs()
            w = torch.softmax(x.masked_fill(hidden, -1e300), -1).masked_fill(hidden, 0.0)
            o[:, h] = w @ v[g]
        outs.append(o)
    o = torch.cat(outs)
    return (o, None, None) if st["append"] else o
