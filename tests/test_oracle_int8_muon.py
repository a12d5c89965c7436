"""Pins of the oracle of the 8-bit base and of the orthogonalised step: hand
cases, invariants, float64 differences, other routes to the same result."""

import numpy as np
import pytest

from oracle import int8 as oi8
from oracle import muon as omu

NS = (3.4445, -4.7750, 2.0315)


def f32(x):
    return np.asarray(x, dtype=np.float32)


def test_record_by_hand():
    # max 127: scale 1, codes are the values rounded, ties to even
    codes, scale = oi8.record(f32([[127, 0.5, 1.5, -0.5, -2.5, 2.5, -126.6, 0.49]]))
    assert scale[0] == 1 and codes.tolist() == [[127, 0, 2, 0, -2, 2, -127, 0]]
    codes, scale = oi8.record(f32([[0, 0, -0.0, 0]]))
    assert scale[0] == 0 and not codes.any()
    codes, scale = oi8.record(f32([[1, np.inf, -3], [1, np.nan, -3]]))
    assert np.isinf(scale[0]) and np.isnan(scale[1]) and not codes.any()
    # the smallest float32: the scale rounds to zero, and so do the codes
    codes, scale = oi8.record(f32([[1e-45, 0, -1e-45]]))
    assert scale[0] == 0 and not codes.any()


def test_record_error_and_range():
    w = f32(np.random.default_rng(0).standard_normal((50, 333)))
    codes, scale = oi8.record(w)
    assert abs(codes).max() == 127 and (abs(codes).max(1) == 127).all()
    off = abs(codes * scale.astype(np.float64)[:, None] - w)
    assert (off <= scale[:, None] * (0.5 + 1e-5)).all()


def test_layer_of_exact_codes_is_the_plain_layer():
    # tokens whose largest value is 127: their codes are the values themselves
    rng = np.random.default_rng(1)
    X = rng.integers(-127, 128, (5, 40)).astype(np.float64)
    X[:, 7] = 127
    W = rng.integers(-127, 128, (9, 40))
    sw = f32(2.0 ** rng.integers(-9, -3, 9))
    A, B = rng.standard_normal((3, 40)), rng.standard_normal((9, 3))
    Y, H = oi8.forward(W, sw, f32(X), A, B, 0.5)
    want = X @ (W * sw[:, None]).T + 0.5 * (X @ A.T) @ B.T
    assert np.allclose(Y, want, rtol=1e-13) and np.allclose(H, X @ A.T, rtol=1e-13)


def test_backward_is_the_gradient_of_the_layer():
    """<dY, Y> is linear in each of X (its rounding passed through), A and B:
    differences are exact but for dY's codes, which move an entry of the
    row by at most half its scale."""
    rng = np.random.default_rng(2)
    M, d, k, r, s = 4, 24, 16, 3, 0.75
    X, dY = f32(rng.standard_normal((M, k))), f32(rng.standard_normal((M, d)))
    W, sw = rng.integers(-127, 128, (d, k)), f32(rng.uniform(0.5, 2, d) / 127)
    A, B = rng.standard_normal((r, k)), rng.standard_normal((d, r))
    dX, dA, dB, se = oi8.backward(W, sw, X, A, B, s, dY)
    Wd = W * sw.astype(np.float64)[:, None]

    def loss(x, a, b):
        return (dY * (x @ Wd.T + s * (x @ a.T) @ b.T)).sum()

    x64, eps = X.astype(np.float64), 1e-4

    def difference(which, at):
        v = [x64, A, B]
        out = []
        for sign in (1, -1):
            t = [y.copy() for y in v]
            t[which][at] += sign * eps
            out.append(loss(*t))
        return (out[0] - out[1]) / (2 * eps)

    for which, g in ((0, dX), (1, dA), (2, dB)):
        for at in np.ndindex(g.shape):
            # dX: each of the d codes of the token off by half a scale
            tol = 0.501 * se[at[0]] * abs(W[:, at[1]]).sum() if which == 0 else 0.0
            assert abs(difference(which, at) - g[at]) <= tol + 1e-8, (which, at)


def test_nan_stays_in_its_row():
    rng = np.random.default_rng(3)
    X = f32(rng.standard_normal((3, 16)))
    W, sw = rng.integers(-127, 128, (8, 16)), f32(np.ones(8))
    clean = oi8.forward(W, sw, X)[0]
    X[1, 4] = np.inf
    Y = oi8.forward(W, sw, X)[0]
    assert np.isnan(Y[1]).all() and np.array_equal(Y[[0, 2]], clean[[0, 2]])


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 9), (6, 40), (40, 6), (12, 12)])
@pytest.mark.parametrize("steps", [0, 1, 5])
def test_iteration_acts_on_singular_values(rows, cols, steps):
    u = np.random.default_rng(rows * 50 + cols).standard_normal((rows, cols))
    x = np.linalg.svd(u, compute_uv=False) / np.linalg.norm(u)
    for _ in range(steps):
        x = NS[0] * x + NS[1] * x ** 3 + NS[2] * x ** 5
    U, _, V = np.linalg.svd(u, full_matrices=False)
    assert np.allclose(omu.orthogonalise(u, NS, steps, 0.0), (U * x) @ V, atol=1e-11)


def test_iteration_brings_singular_values_near_one():
    u = np.random.default_rng(5).standard_normal((16, 300))
    s = np.linalg.svd(omu.orthogonalise(u, NS, 5, 1e-7), compute_uv=False)
    assert s.min() > 0.6 and s.max() < 1.3


def test_small_side_recurrence_is_the_iteration():
    """X_steps = Q X0 with S' = P S P, Q' = P Q on the smaller side alone."""
    u = np.random.default_rng(6).standard_normal((7, 90))
    x0 = u / np.linalg.norm(u)
    S, Q = x0 @ x0.T, np.eye(7)
    for _ in range(5):
        P = NS[0] * np.eye(7) + NS[1] * S + NS[2] * S @ S
        S, Q = P @ S @ P, P @ Q
    assert np.allclose(Q @ x0, omu.orthogonalise(u, NS, 5, 0.0), atol=1e-11)


def test_step_closed_forms():
    kw = dict(beta=0.9, nesterov=True, steps=5, eps=1e-7, scale=2.0, coefficients=NS)
    p = f32(np.random.default_rng(7).standard_normal((2, 3, 8)))
    z = f32(np.zeros((2, 3, 8)))
    # no gradient and no momentum: the decay alone
    q, m, _ = omu.muon_step(p, z, z, lr=0.1, weight_decay=0.5, **kw)
    assert np.allclose(q, 0.95 * p.astype(np.float64)) and not m.any()
    # one row: the update is the row over its norm, times the mapped value 1
    g = f32(np.random.default_rng(8).standard_normal((1, 1, 8)))
    q, m, _ = omu.muon_step(p[:1, :1], z[:1, :1], g, lr=1.0, weight_decay=0.0, **kw)
    x = 1.0
    for _ in range(5):
        x = NS[0] * x + NS[1] * x ** 3 + NS[2] * x ** 5
    want = p[:1, :1] - 2.0 * x * g / np.linalg.norm(g)
    assert np.allclose(q, want, atol=1e-5)
    assert np.array_equal(m, f32(f32(0.1) * g))
