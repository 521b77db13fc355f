"""Test-side helpers of the scored attention tests: cases, the fp64 reference and the bound that roundings allow."""
from __future__ import annotations

import dataclasses
from typing import Optional

import numpy as np
import torch

from oracle import fp8_rows
from oracle.scored import scored_attention
from paged_kv_cache_279_gb300 import workloads as wl
from harness import place_paged, token_slots


@dataclasses.dataclass
class Case:
    lens: list
    Hq: int = 8
    Hkv: int = 2
    D: int = 128
    B: int = 16
    qlens: Optional[list] = None        # None: decode
    dtype: torch.dtype = torch.bfloat16
    softcap: float = 0.0
    alibi: bool = False
    window: int = 0
    prefix: Optional[list] = None
    starts: Optional[list] = None       # per query
    scale: Optional[float] = None
    qmul: float = 2.0
    rows: bool = False                  # row-scaled FP8 cache
    seed: int = 1

    def __post_init__(self):
        S = len(self.lens)
        self.nq = [1 if L else 0 for L in self.lens] if self.qlens is None else list(self.qlens)
        rowsq = [1] * S if self.qlens is None else self.nq   # rows of q per sequence
        self.q_starts = np.concatenate([[0], np.cumsum(rowsq)]).astype(np.int32)
        self.scale = self.D ** -0.5 if self.scale is None else self.scale
        shape = wl.DecodeShape("scored", S, self.Hq, self.Hkv, self.D, self.B, self.dtype)
        counts = [-(-L // self.B) for L in self.lens]
        self.NB = max(1, sum(counts) + 3)
        self.maxB = max(1, max(counts))
        self.tables = wl.random_block_tables(counts, self.NB, self.maxB, self.seed + 1)
        kv = [wl.draw_seq_kv(shape, self.seed, s, L) for s, L in enumerate(self.lens)]
        self.ks, self.vs = [k for k, _ in kv], [v for _, v in kv]
        self.q = (self.qmul * wl.draw_normal((max(1, int(self.q_starts[-1])), self.Hq, self.D), torch.float32,
                                             wl.sub_seed(self.seed, 20))).to(self.dtype)[:int(self.q_starts[-1])]
        self.slopes = np.exp2(-8.0 * np.arange(1, self.Hq + 1) / self.Hq).astype(np.float32) if self.alibi else None
        if self.rows:  # rows of very different sizes, then their values
            r = np.random.default_rng(self.seed + 7)
            self.codes = []
            for i in range(S):
                pair = []
                for x, wide in ((self.ks[i], 1.0), (self.vs[i], 3.0)):
                    f = np.exp(r.uniform(-wide, wide, x.shape[:2]))[..., None]
                    pair.append(fp8_rows.quantise_rows((x.float().numpy() * f).astype(np.float32)) if x.shape[0] else
                                (np.zeros(x.shape, np.uint8), np.zeros(x.shape[:2], np.uint8)))
                self.codes.append(pair)
            self.ks = [torch.from_numpy(fp8_rows.row_values(*p[0])) for p in self.codes]
            self.vs = [torch.from_numpy(fp8_rows.row_values(*p[1])) for p in self.codes]

    # ---- pools -------------------------------------------------------------------------------------------
    def pools(self, fill=float("nan")):
        """Device pools; every slot that no sequence owns holds `fill` (FP8: NaN codes and scale bytes of 255)."""
        if not self.rows:
            kc, vc = place_paged(self.ks, self.vs, self.tables, self.NB, self.B, self.dtype, fill)
            return dict(k_cache=kc.cuda(), v_cache=vc.cuda())
        out = {}
        for j, n in enumerate("kv"):
            c = np.full((self.NB, self.Hkv, self.B, self.D), 0xFF, np.uint8)
            e = np.full((self.NB, self.Hkv, self.B), 0xFF, np.uint8)
            for s, pair in enumerate(self.codes):
                slots = token_slots(self.tables[s], pair[j][1].shape[0], self.B)
                c[slots // self.B, :, slots % self.B] = self.codes[s][j][0]
                e[slots // self.B, :, slots % self.B] = self.codes[s][j][1]
            out[n + "_cache"], out[n + "_scales"] = torch.from_numpy(c).cuda(), torch.from_numpy(e).cuda()
        return out

    def device_args(self):
        i32 = lambda x: None if x is None else torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
        return dict(block_tables=torch.from_numpy(self.tables).cuda(), seq_lens=i32(self.lens),
                    softcap=self.softcap, window=self.window, prefix_lens=i32(self.prefix), key_starts=i32(self.starts),
                    alibi_slopes=None if self.slopes is None else torch.from_numpy(self.slopes).cuda())

    # ---- reference ---------------------------------------------------------------------------------------
    def reference(self):
        """(out, bound) over all query rows.

        The bound counts roundings.  A score is a sum of D products in float32 (at most (D + 16) 2^-24 of scale
        sum |q||k|), and its cap, bias and change of base cost 2^-20 of what they add (the approximate exponential and
        reciprocal are good to 2^-21); a weight is off by twice that and by 2^-8 where it is rounded to bf16 (2^-11 for
        the f16 weights over FP8 codes); sums over n keys by n 2^-24.  Numerator and denominator each take that of
        sum_t w_t |v_t|.  The result is rounded once (half a step: eps / 2 of the type)."""
        outs, tols = [], []
        half = torch.finfo(self.dtype).eps / 2
        weight = 0.0 if self.dtype == torch.float32 else 2.0 ** -11 if self.rows else 2.0 ** -8
        for s, L in enumerate(self.lens):
            n = int(self.q_starts[s + 1] - self.q_starts[s])
            q = self.q[int(self.q_starts[s]):int(self.q_starts[s + 1])].double().numpy()
            k, v = self.ks[s].double().numpy(), self.vs[s].double().numpy()
            if L == 0 or n == 0:
                outs.append(np.zeros(q.shape))
                tols.append(np.zeros(q.shape))
                continue
            st = None if self.starts is None else self.starts[int(self.q_starts[s]):int(self.q_starts[s + 1])]
            o, size = scored_attention(q, k, v, self.scale, self.softcap, self.slopes, self.window,
                                       0 if self.prefix is None else min(max(0, self.prefix[s]), L), st)
            rep = self.Hq // self.Hkv
            a = abs(self.scale) * max(float((np.abs(q[:, h]) @ np.abs(k[:, h // rep]).T).max()) for h in range(self.Hq))
            bias = float(self.slopes.max()) * L if self.slopes is not None else 0.0
            x = (self.D + 16) * 2.0 ** -24 * a + 2.0 ** -20 + 2.0 ** (-20 if self.qlens is None else -18) * self.softcap + 2.0 ** -22 * (bias + a)
            outs.append(o)
            tols.append(2 * (2 * x + weight + L * 2.0 ** -24) * size + half * np.abs(o) * (1 + 2.0 ** -6) + 1e-30)
        return np.concatenate(outs), np.concatenate(tols)

    def check(self, got: torch.Tensor, what=""):
        ref, tol = self.reference()
        g = got.double().cpu().numpy()
        assert g.shape == ref.shape
        assert np.all(np.isfinite(g)), f"{what}: non-finite output"
        over = np.abs(g - ref) - tol
        assert over.max() <= 0, (f"{what}: off by {np.abs(g - ref).flat[over.argmax()]:.3e} at "
                                 f"{np.unravel_index(over.argmax(), ref.shape)}, bound {tol.flat[over.argmax()]:.3e}")
