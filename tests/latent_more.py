"""More of latent attention's cases: tokens whose weight is zero, block tables wider than the contexts."""
import numpy as np
import torch

import latent_cases as lc


def store(c):
    """Writes the rows of a case into its pool (after they were changed)."""
    B = c["B"]
    for s, x in enumerate(c["rows"]):
        p = np.arange(x.shape[0])
        c["cache"][torch.from_numpy(c["tables"][s][p // B].astype(np.int64)), torch.from_numpy(p % B)] = x
    return c


def wide(c, tokens=8192):
    """The case with block tables of at least so many tokens: the longest context there may be is long, so contexts are
    cut into shares and joined, however short they are.  No call may look at the entries behind a context."""
    t = c["tables"]
    extra = max(0, -(-tokens // c["B"]) - t.shape[1])
    return dict(c, tables=np.concatenate([t, np.full((t.shape[0], extra), -1, t.dtype)], 1))


def expected(c, dead, scale=lc.SCALE, terms=None, moves=0):
    """(out, tolerance) with the tokens where dead[s] [H, L] is set left out of every softmax.  The tolerance is that of
    latent_cases.expected, a score's sum over ``terms`` products that are not zero (default: all), ``moves`` times
    the rounding of the reference that weights are taken against, 2^-24 of the largest score each, and weights below
    2^-126 that count as none."""
    D, V, L = c["V"] + 64, c["V"], max(c["lens"])
    terms = D if terms is None else terms
    u, half = 2.0 ** -24, torch.finfo(c["dtype"]).eps / 2
    outs, tols = [], []
    for s, rows in enumerate(c["rows"]):
        rows = rows.double().numpy()
        q = c["q"][int(c["starts"][s]):int(c["starts"][s + 1])].double().numpy()
        n, H, _ = q.shape
        out, tol = np.zeros((n, H, V)), np.full((n, H, V), 1e-37)
        for i in range(n):
            k = rows.shape[0] - n + i + 1  # tokens in sight
            for h in range(H):
                live = ~dead[s][h, :max(k, 0)]
                r = rows[:max(k, 0)][live]
                if r.shape[0] == 0:
                    continue
                x = scale * (r @ q[i, h])
                w = np.exp(x - x.max())
                w /= w.sum()
                out[i, h] = w @ r[:, :V]
                reach = abs(scale) * (np.abs(r) @ np.abs(q[i, h])).max()
                rel = 2 * (reach * (terms + 4) * u + 2.0 ** -21 + (L + 2) * u + moves * u * np.abs(x).max())
                if c["dtype"] == torch.bfloat16:
                    rel += 2 * half
                tol[i, h] += rel * (w @ np.abs(r[:, :V])) + half * np.abs(out[i, h]) + L * 2.0 ** -126 * np.abs(r[:, :V]).max()
        outs.append(out), tols.append(tol)
    return np.concatenate(outs), np.concatenate(tols)


def none_dead(c):
    return [np.zeros((c["H"], x.shape[0]), dtype=bool) for x in c["rows"]]


def check(got, want_tol):
    want, tol = want_tol
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= tol), f"{np.nanmax(err / tol):.3g} of the tolerance, {np.sum(~(err <= tol))} of {err.size} outside"
