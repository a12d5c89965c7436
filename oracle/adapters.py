"""Many LoRA adapters on one frozen base: forward and backward.

CPU oracle -- test infrastructure only (see ``oracle/__init__.py``). Token m
uses adapter ``ids[m]`` when that is in [0, n), else none; per token this is
the layer of ``oracle.lora`` with that token's own A, B and scale, so the
forward and backward are that module's on each adapter's tokens in turn.
"""

from __future__ import annotations

import numpy as np

from . import lora


def tokens_of(ids, n):
    """Token indices per adapter, in batch order, and those without one."""
    ids = np.asarray(ids, dtype=np.int64)
    return [np.flatnonzero(ids == a) for a in range(n)], np.flatnonzero((ids < 0) | (ids >= n))


def forward(Wd, X, A, B, scale, ids):
    """Float64 ``(Y, H)``; H rows of tokens without an adapter are zero."""
    n, r = A.shape[:2]
    Y = X @ Wd.T
    H = np.zeros((X.shape[0], r))
    for a, rows in enumerate(tokens_of(ids, n)[0]):
        if rows.size:
            Y[rows], H[rows] = lora.forward(Wd, X[rows], A[a], B[a], scale[a])
    return Y, H


def backward(Wd, X, A, B, scale, ids, dY):
    """Float64 ``(dX, dA, dB)`` of ``<dY, Y>``."""
    n = A.shape[0]
    dX = dY @ Wd
    dA, dB = np.zeros(A.shape), np.zeros(B.shape)
    for a, rows in enumerate(tokens_of(ids, n)[0]):
        if rows.size:
            dX[rows], dA[a], dB[a], _ = lora.backward(Wd, X[rows], A[a], B[a], scale[a], dY[rows])
    return dX, dA, dB
