"""Orthogonalised momentum step of the LoRA matrices.

CPU oracle -- test infrastructure only (see ``oracle/__init__.py``). Per matrix,
in float64 except for the momentum, which is state::

    m' = fl(fl(beta * m) + fl(c1 * g))          c1 = fl32(1 - beta)
    u  = fl(fl(c1 * g) + fl(beta * m'))         (nesterov), or m'
    X0 = u / (|u|_F + eps)
    X  = a X + (b (X X^T) + c (X X^T)^2) X      `steps` times
    p' = p - lr (scale X + weight_decay p)

The iteration is run as written, on the matrix itself, in float64.
"""

from __future__ import annotations

import numpy as np

F32 = np.float32


def update_matrix(m, g, beta, nesterov):
    """``(m', u)`` in float32, each operation rounded once; g float32-valued."""
    b, c1 = F32(beta), F32(1.0 - float(beta))
    m, g = np.asarray(m, dtype=F32), np.asarray(g, dtype=F32)
    with np.errstate(all="ignore"):
        m1 = ((b * m).astype(F32) + (c1 * g).astype(F32)).astype(F32)
        u = ((c1 * g).astype(F32) + (b * m1).astype(F32)).astype(F32) if nesterov else m1
    return m1, u


def orthogonalise(u, coefficients, steps, eps):
    """Newton-Schulz iteration of one matrix in float64."""
    a, b, c = coefficients
    x = np.asarray(u, dtype=np.float64)
    x = x / (np.sqrt((x * x).sum()) + eps)
    for _ in range(steps):
        s = x @ x.T if x.shape[0] <= x.shape[1] else x.T @ x
        poly = b * s + c * (s @ s)
        x = a * x + (poly @ x if x.shape[0] <= x.shape[1] else x @ poly)
    return x


def muon_step(p, m, g, *, lr, beta, weight_decay, nesterov, steps, eps, scale, coefficients):
    """One step on n x rows x cols arrays. Returns ``(p' float64, m' float32,
    update float64)``, the update being scale X + weight_decay p."""
    m1, u = update_matrix(m, g, beta, nesterov)
    p = np.asarray(p, dtype=np.float64)
    d = np.stack([scale * orthogonalise(x, coefficients, steps, eps) for x in u])
    d = d + weight_decay * p
    return p - lr * d, m1, d
