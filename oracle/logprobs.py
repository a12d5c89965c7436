"""Log probabilities of given tokens, entropy, best alternatives, gradient.

CPU oracle -- test infrastructure only (see ``oracle/__init__.py``). Softmax
in float64 from its definition, row by row; the special rows (nothing but
-inf, an infinity or NaN, a target outside the vocabulary) as
``include/qlora_logprobs.h`` states them.
"""

from __future__ import annotations

import numpy as np


def row(x):
    """``(logp, p, entropy)`` of one row of logits in float64."""
    x = np.asarray(x, dtype=np.float64)
    if np.isnan(x).any() or np.isposinf(x).any():
        return np.full_like(x, np.nan), np.full_like(x, np.nan), np.nan
    if np.isneginf(x).all():
        return x.copy(), np.zeros_like(x), 0.0
    t = x - x.max()
    logp = t - np.log(np.exp(t).sum())
    p = np.exp(logp)
    on = p > 0
    return logp, p, -(p[on] * logp[on]).sum()


def top(x, n):
    """Indices of the n largest: NaN first, then by value descending, equal
    values (the two zeros among them) by index."""
    x = np.asarray(x, dtype=np.float64) + 0.0
    return np.lexsort((np.arange(x.size), -np.where(np.isnan(x), np.inf, x), ~np.isnan(x)))[:n]


def forward(x, targets, n=0):
    """``(logprob, entropy, top_logprobs, top_ids)``."""
    N, V = x.shape
    lp, ent = np.zeros(N), np.zeros(N)
    tl, ti = np.zeros((N, n)), np.zeros((N, n), dtype=np.int64)
    for i in range(N):
        logp, _, ent[i] = row(x[i])
        if 0 <= targets[i] < V:
            lp[i] = logp[targets[i]]
        ti[i] = top(x[i], n)
        tl[i] = logp[ti[i]]
    return lp, ent, tl, ti


def backward(x, targets, g, e=None):
    """Gradient of ``sum_i g_i logprob_i + e_i entropy_i``."""
    N, V = x.shape
    dx = np.zeros((N, V))
    for i in range(N):
        gi = g[i] if 0 <= targets[i] < V else 0.0
        ei = 0.0 if e is None else e[i]
        if gi == 0.0 and ei == 0.0:
            continue
        logp, p, ent = row(x[i])
        if np.isneginf(x[i]).all():
            continue
        d = np.zeros(V)
        if gi != 0.0:
            d[targets[i]] = gi
        with np.errstate(invalid="ignore"):
            plogp = np.where(p == 0, 0.0, p * logp)
        dx[i] = d - gi * p - ei * (plogp + p * ent)
    return dx
