"""Float64 CPU oracle of sampling and of the embedding -- TEST INFRASTRUCTURE
ONLY, as the rest of this package.

Written from the definitions, plainly: a row's columns are sorted by falling
logit, equal ones by rising number; top-k, top-p (of what top-k keeps) and
min-p each keep a prefix; the draw walks the kept columns by number.
"""
from __future__ import annotations

import numpy as np


def sample_row(x, u, t=1.0, k=0, p=1.0, m=0.0):
    """(token, logp, kept, margin): margin is how far, in parts of the kept sum, the draw and top_p's border are
    from the next weight's edge -- what an error in the weights would have to pass to change the answer."""
    x = np.asarray(x, np.float64)
    allowed = np.flatnonzero(x > -np.inf)
    if not allowed.size:
        return -1, 0.0, 0, 1.0
    if t < 1e-6:
        t, k = 1.0, 1
    z = (x[allowed] - x[allowed].max()) / t
    w = np.exp(z)
    order = np.lexsort((allowed, -x[allowed]))
    margin = 1.0
    n = order.size
    if k > 0:
        n = min(n, int(k))
    if p < 1.0:
        run = np.cumsum(w[order[:n]])
        goal = p * run[-1]
        margin = np.abs(run[:-1] / run[-1] - p).min() if n > 1 and p > 0 else 1.0
        n = 1 + int(np.searchsorted(run, goal)) if p > 0 else 1
    if m > 0.0:
        n = min(n, max(1, int((w[order] >= min(m, 1.0)).sum())))
    kept = np.sort(order[:n])
    run = np.cumsum(w[kept])
    at = min(n - 1, int(np.searchsorted(run, u * run[-1], side="right")))
    if n > 1:
        margin = min(margin, np.abs(run[:-1] / run[-1] - u).min())
    return int(allowed[kept[at]]), float(z[kept[at]] - np.log(w.sum())), n, float(margin)


def sample(x, u, t=1.0, k=0, p=1.0, m=0.0):
    """sample_row of each row; the settings are numbers or [rows]."""
    rows = len(u)
    each = [np.broadcast_to(np.asarray(v, np.float64), (rows,)) for v in (t, k, p, m)]
    out = [sample_row(x[r], float(u[r]), *(float(v[r]) for v in each)) for r in range(rows)]
    return tuple(np.array([o[i] for o in out]) for i in range(4))


def lookup(table, ids, scale=1.0):
    table, ids = np.asarray(table, np.float64), np.asarray(ids)
    out = np.zeros((ids.size, table.shape[1]))
    there = (ids >= 0) & (ids < table.shape[0])
    out[there] = table[ids[there]] * scale
    return out


def lookup_grad(dy, ids, vocab, scale=1.0):
    """(gradient, sum of the terms' sizes, counts)."""
    dy, ids = np.asarray(dy, np.float64), np.asarray(ids)
    there = np.flatnonzero((ids >= 0) & (ids < vocab))
    grad, size = np.zeros((vocab, dy.shape[1])), np.zeros((vocab, dy.shape[1]))
    np.add.at(grad, ids[there], dy[there] * scale)
    np.add.at(size, ids[there], np.abs(dy[there] * scale))
    return grad, size, np.bincount(ids[there], minlength=vocab)
