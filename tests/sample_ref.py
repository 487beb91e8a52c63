"""The token choice in float64, by sorting, and how near its draw lies to a border."""

import numpy as np


def sample(row, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, log probability, margin) of one row of float64 logits without NaN; margin: how far the nearest border of a
    decision lies, in units of the largest e."""
    order = np.argsort(-row, kind="stable")
    top = row[order[0]]
    if top == -np.inf:
        return -1, -np.inf, 1.0
    if not temperature > 0:
        return int(order[0]), 0.0, 1.0
    with np.errstate(invalid="ignore", under="ignore"):
        z = np.where(row[order] == top, 0.0, (row[order] - top) / temperature)
    z[np.isnan(z)] = -np.inf
    e = np.where(row[order] > -np.inf, np.exp(z), 0.0)
    keep = len(e) if top_k <= 0 else min(int(top_k), len(e))
    least = min(max(min_p, 0.0), 1.0) if min_p == min_p else 0.0
    # e of the top's equals is 1 on both sides, and compares exactly.  Where nothing else is kept sums are whole numbers
    # below 2^20, and their products with shares of 24 bits exact: no border is near.
    near = np.abs(e[:keep][e[:keep] < 1] - least)
    margin = float(near.min()) if least > 0 and len(near) else 1.0
    e = e[:keep]
    e = e[e >= least]
    whole = bool((e == 1).all()) and all(v == np.float32(v) for v in (top_p, u))
    upto = np.cumsum(e)
    if top_p < 1:
        want = max(top_p, 0.0) * upto[-1]
        n = int(np.searchsorted(upto, want)) + 1
        near = upto[:-1]
        if top_p > 0 and len(near) and not whole:
            margin = min(margin, float(np.abs(near - want).min()))
        e, upto = e[:min(n, len(e))], upto[:min(n, len(e))]
    want = min(max(u, 0.0), 1.0) * upto[-1]
    at = min(int(np.searchsorted(upto, want, side="right")), len(e) - 1)
    if len(e) > 1 and 0 < u < 1 and not whole:
        margin = min(margin, float(np.abs(upto[:-1] - want).min()))
    return int(order[at]), float(z[at] - np.log(upto[-1])), margin
