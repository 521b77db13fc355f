"""Cases of the rotary position and latent attention operators, for timing and checking them.

Five operators of a paged KV cache:

* rotate: rotary_embed -- queries or keys rotated by their positions, half or interleaved pairs, the whole head or part
  of it, frequencies as they are or scaled for long contexts;
* write: kv_cache_write_rotary -- new keys rotated on their way into the paged cache, values stored beside them, the
  queries rotated in the same call;
* latent_write: latent_cache_write -- one row a token, shared by all heads, [latent | rotated key part], stored in its
  paged cache, and the rotary part of the queries rotated into their place;
* decode: paged_latent_attention_decode -- one query a sequence over that cache;
* multi: paged_latent_attention_multi_token -- several causal queries a sequence over it.

Rotation at position p, pair i of R / 2 with frequency f_i, amplitude a (c = a cos(p f_i), s = a sin(p f_i)):
    y1 = x1 c - x2 s,  y2 = x2 c + x1 s      pairs (i, i + R / 2), or (2 i, 2 i + 1) where interleaved
Latent attention of the query at position p, with c_t = [latent_t | key part_t] the row of token t <= p:
    out = sum_t softmax_t(scale * q . c_t) latent_t

With ``own`` false, run() computes the plain forms in elementary torch operations; with ``own`` true it makes the
calls of the framework.
"""
import math
import random

import torch

own = False
DEV = "cuda"
ROPE = 64  # entries of a latent row's rotary part


# ---------------------------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------------------------
def _rotate(name, **k):
    return dict({"op": "rotate", "tokens": 64, "heads": 32, "head_dim": 128, "rotary": 128, "offset": 0, "interleaved": False,
                 "scaling": "none", "far": 16000, "dtype": "bf16"}, **k, name=name)


def _write(name, **k):
    return dict({"op": "write", "tokens": 64, "heads": 32, "kv_heads": 8, "head_dim": 128, "rotary": 128, "offset": 0,
                 "block": 16, "interleaved": False, "scaling": "none", "far": 16000, "dtype": "bf16"}, **k, name=name)


def _latent_write(name, **k):
    return dict({"op": "latent_write", "tokens": 64, "heads": 32, "latent": 512, "rotary": ROPE, "block": 16, "interleaved": True,
                 "scaling": "parts", "far": 16000, "dtype": "bf16"}, **k, name=name)


def _attend(name, op, **k):
    c = {"op": op, "seqs": 64, "len_lo": 64, "len_hi": 2048, "heads": 32, "latent": 512, "block": 16, "dtype": "bf16"}
    if op == "multi":
        c["queries"] = 5
    return dict(c, **k, name=name)


def listed():
    return [
        # the queries of one decode step of 64 sequences: latency
        _rotate("rotate 64 tokens"),
        # the queries of a prefill batch, half of each head rotated in interleaved pairs, long-context frequencies
        _rotate("rotate 16384 tokens interleaved half", tokens=16384, rotary=64, interleaved=True, scaling="parts"),
        # one decode step's queries, keys and values, slices of one projection
        _write("write 64 tokens"),
        # the prompts of a prefill batch, their number no multiple of anything
        _write("write 16001 tokens", tokens=16001, scaling="linear"),
        # one decode step's latent rows
        _latent_write("latent write 64 tokens"),
        # the latent rows of a prefill batch
        _latent_write("latent write 16001 tokens", tokens=16001, block=32),
        # four short sequences in float32: the smallest attention call
        _attend("decode tiny float32", "decode", seqs=4, len_lo=1, len_hi=100, heads=4, dtype="f32"),
        # the serving step: 64 sequences of mixed lengths
        _attend("decode 64 x 64..2048", "decode"),
        # long contexts, twice the heads
        _attend("decode 8 x 16000", "decode", seqs=8, len_lo=16000, len_hi=16000, heads=64),
        # five drafted tokens a sequence to verify
        _attend("multi 64 x 5", "multi"),
        # a prefill chunk at the end of 4096 tokens
        _attend("multi 8 x 512 of 4096", "multi", seqs=8, len_lo=4096, len_hi=4096, queries=512),
        # whole prompts, ragged
        _attend("multi 4 prompts", "multi", seqs=4, len_lo=3200, len_hi=4000, queries=4000, heads=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "write", "latent_write", "decode", "decode", "decode", "multi", "multi", "multi"])
    if op in ("rotate", "write"):
        D = rng.choice([64, 128])
        R = rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= D] + [D])
        c = {"op": op, "head_dim": D, "rotary": R, "offset": rng.choice([0, 0, D - R]), "interleaved": rng.random() < 0.5,
             "scaling": rng.choice(["none", "linear", "parts"]), "far": _log(rng, 100, 1000000),
             "dtype": rng.choice(["bf16", "bf16", "f32"])}
        if op == "rotate":
            c["heads"] = rng.choice([1, 3, 8, 16, 32, 40, 64])
        else:
            c["kv_heads"] = rng.choice([1, 2, 3, 4, 8])
            c["heads"] = c["kv_heads"] * rng.randint(1, 8)
            c["block"] = rng.choice([8, 16, 32])
        c["tokens"] = max(1, min(_log(rng, 1, 40000), 16384 * 32 // c["heads"], 16384 * 8 // c.get("kv_heads", 8)))
        return c
    c = {"op": op, "heads": rng.choice([1, 2, 4, 8, 12, 16, 20, 24, 32, 40, 48, 64, 96, 128]), "latent": rng.choice([256, 512, 512]),
         "block": rng.choice([8, 16, 32, 64]), "dtype": "bf16"}
    if op == "latent_write":
        c.update({"rotary": ROPE, "interleaved": rng.random() < 0.5, "scaling": rng.choice(["none", "linear", "parts"]),
                  "far": _log(rng, 100, 1000000), "dtype": rng.choice(["bf16", "bf16", "f32"])})
        c["tokens"] = max(1, min(_log(rng, 1, 40000), 16001 * 32 // c["heads"]))
        return c
    if op == "decode":
        c["dtype"] = rng.choice(["bf16", "bf16", "bf16", "f32"])
    c["seqs"] = _log(rng, 1, 64)
    c["len_hi"] = _log(rng, 1, min(16000, (2048 if c["dtype"] == "f32" else 65536) // c["seqs"]))
    c["len_lo"] = max(1, _log(rng, max(1, c["len_hi"] // 30), c["len_hi"]))
    if op == "multi":
        most = max(1, 2 ** 28 // (c["seqs"] * c["len_hi"] * c["heads"]))
        c["queries"] = _log(rng, 1, min(most, c["len_hi"], 2048))
    return c


def _plan(case, seed):
    """Lengths and query counts of an attention case.  The lengths are the case's own, their order the seed's: every seed's
    batch holds as many tokens and blocks."""
    r = random.Random("%d to %d" % (case["len_lo"], case["len_hi"]))
    lens = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["seqs"])]
    random.Random("%d plan" % seed).shuffle(lens)
    return lens, [min(case.get("queries", 1), L) for L in lens]


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "rotate":  # every entry read and written; a position (4 bytes) a token
        n = case["tokens"] * case["heads"]
        return {"bytes": n * case["head_dim"] * 2 * size + case["tokens"] * 4, "flops": n * case["rotary"] * 3}
    if case["op"] == "write":  # and a slot (8 bytes)
        T, H, K = case["tokens"], case["heads"], case["kv_heads"]
        return {"bytes": T * (H + 2 * K) * case["head_dim"] * 2 * size + T * 12, "flops": T * (H + K) * case["rotary"] * 3}
    if case["op"] == "latent_write":
        T, H = case["tokens"], case["heads"]
        return {"bytes": T * (case["latent"] + ROPE + H * ROPE) * 2 * size + T * 12, "flops": T * (H + 1) * ROPE * 3}
    lens, nq = _plan(case, 0)
    D, V, H = case["latent"] + ROPE, case["latent"], case["heads"]
    pairs = sum(n * L - n * (n - 1) // 2 for L, n in zip(lens, nq))
    return {"bytes": (sum(lens) * D + sum(nq) * H * (D + V)) * size, "flops": 2 * (D + V) * H * pairs}


# ---------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------
def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _frequencies(case):
    """Radians per position, float64 [R / 2]: powers of 10000; all divided by 4; or, by parts, those that turn less than
    once in 4096 positions divided by 8, those that turn 32 times or more as they are, a ramp between."""
    R = case["rotary"]
    f = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    if case["scaling"] == "linear":
        f = f / 4.0
    elif case["scaling"] == "parts":
        w = ((4096.0 * f / (2.0 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
        f = f * (w + (1.0 - w) / 8.0)
    return f.to(DEV)


def _slots(case, gen):
    """(slots, blocks of the pool): consecutive positions of contexts whose blocks lie anywhere in the pool."""
    T, B = case["tokens"], case["block"]
    used = -(-T // B)
    NB = used + used // 10 + 1
    blocks = torch.randperm(NB, generator=gen, device=DEV)[:used]
    at = torch.arange(T, device=DEV)
    return blocks[at // B] * B + at % B, NB


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt = _dtype(case)
    normal = lambda *shape: torch.randn(shape, generator=gen, device=DEV).to(dt)  # noqa: E731
    st = {"case": case}
    if "tokens" in case:
        T = case["tokens"]
        st["freqs"] = _frequencies(case)
        st["amplitude"] = 0.1 * math.log(8.0) + 1.0 if case["scaling"] == "parts" else 1.0
        # a chunk of a few contexts: runs of consecutive positions up to the farthest
        start = torch.randint(0, case["far"], (1 + T // 1000,), generator=gen, device=DEV)
        at = torch.arange(T, device=DEV)
        st["positions"] = (start[at // 1000] + at % 1000).to(torch.int32)
        H = case["heads"]
        if case["op"] == "rotate":
            st["x"] = normal(T, H, case["head_dim"])
            return st
        st["slots"], NB = _slots(case, gen)
        if case["op"] == "write":
            K, D = case["kv_heads"], case["head_dim"]
            qkv = normal(T, H + 2 * K, D)  # one projection's output
            st["q"], st["k"], st["v"] = qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:]
            st["kc"] = torch.zeros((NB, K, case["block"], D), dtype=dt, device=DEV)
            st["vc"] = torch.zeros_like(st["kc"])
        else:
            rows = normal(T, case["latent"] + ROPE)  # one projection's output
            st["latent"], st["k_rope"] = rows[:, :case["latent"]], rows[:, case["latent"]:]
            st["q_rope"] = normal(T, H, ROPE)
            st["q"] = torch.zeros((T, H, case["latent"] + ROPE), dtype=dt, device=DEV)  # its latent part comes from elsewhere
            st["cache"] = torch.zeros((NB, case["block"], case["latent"] + ROPE), dtype=dt, device=DEV)
        return st
    lens, nq = _plan(case, seed)
    B, D, H = case["block"], case["latent"] + ROPE, case["heads"]
    counts = [-(-L // B) for L in lens]
    NB = sum(counts) + sum(counts) // 10 + 1
    ids = torch.randperm(NB, generator=gen, device=DEV).to(torch.int32).cpu()
    tables = torch.zeros((len(lens), max(counts)), dtype=torch.int32)
    at = 0
    for s, n in enumerate(counts):
        tables[s, :n] = ids[at:at + n]
        at += n
    st["tables"], st["lens"] = tables.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    st["q_starts"] = torch.tensor([0] + nq).cumsum(0).to(torch.int32).to(DEV)
    st["max_q"], st["max_len"] = max(nq), max(lens)
    st["scale"] = 1.0 / math.sqrt(192.0)
    st["cache"] = normal(NB, B, D)
    st["q"] = normal(sum(nq), H, D)
    return st


# ---------------------------------------------------------------------------------------------------------------
# The operators
# ---------------------------------------------------------------------------------------------------------------
def run(st):
    op = st["case"]["op"]
    if own:
        return {"rotate": _own_rotate, "write": _own_write, "latent_write": _own_latent_write, "decode": _own_decode,
                "multi": _own_multi}[op](st)
    return {"rotate": _plain_rotate, "write": _plain_write, "latent_write": _plain_latent_write, "decode": _plain_attend,
            "multi": _plain_attend}[op](st)


def _own_rotate(st):
    import paged_kv_cache_279_gb300 as pkv
    c = st["case"]
    return pkv.rotary_embed(torch.empty_like(st["x"]), st["x"], st["positions"], st["freqs"], amplitude=st["amplitude"],
                            interleaved=c["interleaved"], offset=c["offset"])


def _own_write(st):
    import paged_kv_cache_279_gb300 as pkv
    c = st["case"]
    q_out = torch.empty(st["q"].shape, dtype=st["q"].dtype, device=DEV)
    pkv.kv_cache_write_rotary(st["k"], st["v"], st["kc"], st["vc"], st["slots"], st["positions"], st["freqs"], q=st["q"],
                              q_out=q_out, amplitude=st["amplitude"], interleaved=c["interleaved"], offset=c["offset"])
    return q_out, st["kc"], st["vc"]


def _own_latent_write(st):
    import paged_kv_cache_279_gb300 as pkv
    c = st["case"]
    pkv.latent_cache_write(st["latent"], st["k_rope"], st["cache"], st["slots"], st["positions"], st["freqs"],
                           q_rope=st["q_rope"], q_out=st["q"][..., c["latent"]:], amplitude=st["amplitude"],
                           interleaved=c["interleaved"])
    return st["cache"], st["q"]


def _own_decode(st):
    import paged_kv_cache_279_gb300 as pkv
    q = st["q"]
    out = torch.empty(q.shape[:2] + (st["case"]["latent"],), dtype=q.dtype, device=DEV)
    return pkv.paged_latent_attention_decode(out, q, st["cache"], st["tables"], st["lens"], st["scale"], st["max_len"])


def _own_multi(st):
    import paged_kv_cache_279_gb300 as pkv
    q = st["q"]
    out = torch.empty(q.shape[:2] + (st["case"]["latent"],), dtype=q.dtype, device=DEV)
    return pkv.paged_latent_attention_multi_token(out, q, st["cache"], st["tables"], st["lens"], st["q_starts"], st["scale"],
                                                  st["max_q"], st["max_len"])


def _turned(st, x, offset):
    """Rows x [T, H, D] with the entries from ``offset`` on rotated, rounded once; angles in 64 bits."""
    c = st["case"]
    R = c["rotary"]
    angle = st["positions"].double()[:, None] * st["freqs"]
    cos, sin = ((st["amplitude"] * f(angle)).float()[:, None] for f in (torch.cos, torch.sin))
    y = x.float()
    part = y[..., offset:offset + R]
    if c["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = part[..., :R // 2], part[..., R // 2:]
        part = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y[..., :offset], part, y[..., offset + R:]], -1).to(x.dtype)


def _plain_rotate(st):
    return _turned(st, st["x"], st["case"]["offset"])


def _plain_write(st):
    c = st["case"]
    blk, off = st["slots"] // c["block"], st["slots"] % c["block"]
    st["kc"][blk, :, off] = _turned(st, st["k"], c["offset"])
    st["vc"][blk, :, off] = st["v"]
    return _turned(st, st["q"], c["offset"]), st["kc"], st["vc"]


def _plain_latent_write(st):
    c = st["case"]
    blk, off = st["slots"] // c["block"], st["slots"] % c["block"]
    st["cache"][blk, off] = torch.cat([st["latent"], _turned(st, st["k_rope"][:, None], 0)[:, 0]], -1)
    st["q"][..., c["latent"]:] = _turned(st, st["q_rope"], 0)
    return st["cache"], st["q"]


def _plain_attend(st):
    """The whole matrix of scores in float32, masked."""
    c = st["case"]
    V, H = c["latent"], c["heads"]
    lens, q0, Q = st["lens"].long(), st["q_starts"].long(), st["max_q"]
    rows = st["cache"][st["tables"].long()].flatten(1, 2)[:, :st["max_len"]].float()       # [S, L, D]
    t = torch.arange(rows.shape[1], device=DEV)
    rows = rows.masked_fill((t >= lens[:, None])[:, :, None], 0.0)
    S, L, D = rows.shape
    nq = q0[1:] - q0[:-1]
    i = torch.arange(Q, device=DEV)
    live = i < nq[:, None]                                                                 # [S, Q]
    q = st["q"][torch.where(live, q0[:-1, None] + i, 0)].float().reshape(S, Q * H, D)
    x = (torch.bmm(q, rows.transpose(1, 2)) * st["scale"]).reshape(S, Q, H, L)
    p = (lens - nq)[:, None] + i
    x = x.masked_fill((t > p[:, :, None])[:, :, None], float("-inf"))
    w = torch.exp(x - x.amax(-1, keepdim=True))
    w = w / w.sum(-1, keepdim=True)
    o = torch.bmm(w.reshape(S, Q * H, L), rows[..., :V]).reshape(S, Q, H, V)
    return o[live].to(st["q"].dtype)


# ---------------------------------------------------------------------------------------------------------------
# The definition, in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def _exact_turn(st, x, offset):
    """The rotation as a product of complex numbers."""
    c = st["case"]
    R = c["rotary"]
    phase = torch.outer(st["positions"].double(), st["freqs"])
    turn = torch.polar(torch.full_like(phase, st["amplitude"]), phase)[:, None]
    y = x.double()
    n = torch.arange(R // 2, device=DEV)
    first, second = (offset + 2 * n, offset + 2 * n + 1) if c["interleaved"] else (offset + n, offset + R // 2 + n)
    z = torch.complex(y[..., first], y[..., second]) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rotate":
        return _exact_turn(st, st["x"], case["offset"])
    if "tokens" in case:
        at = (torch.div(st["slots"], case["block"], rounding_mode="floor"), st["slots"] % case["block"])
        if case["op"] == "write":
            kc, vc = (torch.zeros(st["kc"].shape, dtype=torch.float64, device=DEV) for _ in range(2))
            kc.transpose(1, 2)[at] = _exact_turn(st, st["k"], case["offset"])
            vc.transpose(1, 2)[at] = st["v"].double()
            return _exact_turn(st, st["q"], case["offset"]), kc, vc
        cache = torch.zeros(st["cache"].shape, dtype=torch.float64, device=DEV)
        row = torch.empty((case["tokens"], cache.shape[2]), dtype=torch.float64, device=DEV)
        row[:, :case["latent"]] = st["latent"]
        row[:, case["latent"]:] = _exact_turn(st, st["k_rope"].unsqueeze(1), 0).squeeze(1)
        cache[at] = row
        q = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
        q[..., case["latent"]:] = _exact_turn(st, st["q_rope"], 0)
        return cache, q
    q0, outs = st["q_starts"].tolist(), []
    for s, L in enumerate(st["lens"].tolist()):  # each sequence by itself, its context laid out in order
        rows = st["cache"][st["tables"][s, :-(-L // case["block"])].long()].flatten(0, 1)[:L].double()
        q = st["q"][q0[s]:q0[s + 1]].double()
        n = q.shape[0]
        hidden = torch.arange(L, device=DEV)[None] > torch.arange(L - n, L, device=DEV)[:, None]
        o = torch.empty((n, case["heads"], case["latent"]), dtype=torch.float64, device=DEV)
        for h in range(case["heads"]):
            w = torch.softmax((q[:, h] @ rows.T * st["scale"]).masked_fill(hidden, float("-inf")), -1)
            o[:, h] = w @ rows[:, :case["latent"]]
        outs.append(o)
    return torch.cat(outs)
