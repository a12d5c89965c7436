"""8-bit integer base: records by row, the layer's forward and its backward.

CPU oracle -- test infrastructure only (see ``oracle/__init__.py``). Row i of a
matrix has the scale s_i = max|w| / 127, correctly rounded to float32, and the
codes w / s_i, the quotient correctly rounded to float32, then to the nearest
whole number (ties to even) and held in [-127, 127]; a zero scale has zero
codes. The codes are decisions and follow these float32 roundings; everything
else is float64. A scale that is not finite makes the row's products NaN.
"""

from __future__ import annotations

import numpy as np

F32 = np.float32


def record(w):
    """``(codes int64, scale float32)`` of the rows of ``w`` (float32 values)."""
    w = np.asarray(w, dtype=F32)
    with np.errstate(all="ignore"):
        scale = (np.abs(w).max(axis=1) / F32(127)).astype(F32)   # max keeps a NaN
        t = np.rint((w / scale[:, None]).astype(F32)).astype(np.float64)
    t[np.isnan(t)] = 0.0
    codes = np.clip(t, -127, 127).astype(np.int64)
    codes[scale == 0] = 0
    return codes, scale


def _product(a, b):
    """Product of whole numbers, exact in float64 (sums below 2^53)."""
    return a.astype(np.float64) @ b.astype(np.float64)


def forward(codes, scale, X, A=None, B=None, s=0.0):
    """Float64 ``(Y, H)`` of float32-valued tokens ``X``."""
    xq, sx = record(X)
    with np.errstate(invalid="ignore"):
        Y = _product(xq, codes.T) * sx.astype(np.float64)[:, None] * \
            scale.astype(np.float64)
    if A is None:
        return Y, None
    H = X.astype(np.float64) @ A.T
    return Y + s * (H @ B.T), H


def backward(codes, scale, X, A, B, s, dY):
    """Float64 ``(dX, dA, dB, se)``; se: the float32 scales of dY's rows."""
    with np.errstate(all="ignore"):
        e = (np.asarray(dY, dtype=F32) * np.asarray(scale, dtype=F32)).astype(F32)
    eq, se = record(e)
    with np.errstate(invalid="ignore"):
        dX = _product(eq, codes) * se.astype(np.float64)[:, None]
    if A is None:
        return dX, None, None, se
    dY, X = np.asarray(dY, dtype=np.float64), np.asarray(X, dtype=np.float64)
    G = dY @ B
    return dX + s * (G @ A), s * (G.T @ X), s * (dY.T @ (X @ A.T)), se
