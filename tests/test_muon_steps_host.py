"""Step counts of the orthogonalised step (no GPU, nothing launched): counts at
which rounding has grown past use are refused, by the coefficients."""

import ctypes

import numpy as np
import pytest

from bit_nf4_quantized_19_amd import ops
from oracle import muon as omu

DEFAULT = (3.4445, -4.7750, 2.0315)
#: coefficients and the most steps that a^(2 steps) <= 2^36 leaves
LIMITS = [(DEFAULT, 10), ((1.5, -0.5, 0.0), 30), ((15 / 8, -10 / 8, 3 / 8), 19),
          ((2.0, -1.5, 0.5), 18), ((-2.0, 1.5, -0.5), 18), ((1.0, -0.5, 0.0), 32),
          ((0.5, 0.1, 0.1), 32), ((0.0, 1.0, 0.0), 32), ((1e6, -1e6, 1.0), 1),
          ((1e300, 0.0, 0.0), 1)]


def status(coefficients, steps, rows=16, cols=64):
    P = 0x100000   # neither device nor page-locked memory: refused after the counts
    hp = ops.MuonHParamsC(0.02, 0.9, 0.0, 1e-7, 1.0, *coefficients, steps, 1)
    return ops.lib().qlora_muon_step(P, P, P, P, 2, rows, cols, ctypes.addressof(hp), P, 1 << 50,
                                     None)


@pytest.mark.parametrize("coefficients,most", LIMITS)
def test_counts_by_coefficients(coefficients, most):
    for steps in range(33):
        want = ops.QLORA_ERR_INVALID_ARG if steps <= most else ops.QLORA_ERR_UNSUPPORTED
        assert status(coefficients, steps) == want, steps
    assert status(coefficients, 33) == status(coefficients, -1) == ops.QLORA_ERR_INVALID_ARG
    assert most == 32 or status(coefficients, most + 1, 128, 200) == ops.QLORA_ERR_UNSUPPORTED


def small_matrices(u, coefficients, steps):
    """The update as the library forms it: S and Q = P .. P carried in float64."""
    a, b, c = coefficients
    u = u.astype(np.float64)
    S, Q = u @ u.T, np.eye(u.shape[0])
    inv = 1 / np.sqrt(np.trace(S))
    S = S * inv * inv
    for _ in range(steps):
        P = a * np.eye(u.shape[0]) + b * S + c * (S @ S)
        Q, S = P @ Q, P @ (P @ S)
    return inv * Q @ u


def updates():
    rng = np.random.default_rng(3)
    yield np.outer(rng.standard_normal(16), rng.standard_normal(256))
    yield rng.standard_normal((32, 4)) @ rng.standard_normal((4, 256))
    v = np.zeros((16, 256))
    v[:, :3] = rng.standard_normal((16, 3))
    yield v
    v = rng.integers(-3, 4, (32, 200)).astype(float)
    v[16:] = v[:16]
    yield v
    # singular values over eight decades, where the gain is steepest in S
    q1, _ = np.linalg.qr(rng.standard_normal((16, 16)))
    q2, _ = np.linalg.qr(rng.standard_normal((256, 16)))
    yield (q1 * np.logspace(0, -8, 16)) @ q2.T


@pytest.mark.parametrize("coefficients,most", [x for x in LIMITS if 1 < abs(x[0][0]) < 1e5])
def test_accepted_counts_stay_with_the_iteration(coefficients, most):
    """S's roundings, a few 2^-53 of its largest eigenvalue, move the update of
    a direction by at most their size times the gain's slope and the direction's
    singular value, at most a^(2 steps): 16 * 2^(36 - 53) for the few."""
    for u in updates():
        u = u.astype(np.float32)
        for steps in (most // 2, most):
            want = omu.orthogonalise(u, coefficients, steps, 0.0)
            off = np.linalg.norm(small_matrices(u, coefficients, steps) - want)
            assert off <= 16 * abs(coefficients[0]) ** (2 * steps) * 2.0 ** -53, (steps, off)


@pytest.mark.parametrize("rows,cols", [(1, 1), (16, 64), (16, 4096), (11008, 12), (64, 8192),
                                       (128, 129), (130, 100), (4, 1 << 20)])
def test_workspace_sizes_do_not_fall(rows, cols):
    """With more matrices, a longer or a wider one: the workspace of the largest
    serves them all."""
    size = lambda *s: ops.lib().qlora_muon_workspace_bytes(*s)   # noqa: E731
    by_n = [size(n, rows, cols) for n in range(1, 2100)] + [size(65535, rows, cols)]
    assert all(a <= b for a, b in zip(by_n, by_n[1:]))
    for n in (1, 7, 600, 2000):
        long = [size(n, rows, cols + c) if cols >= rows else size(n, rows + c, cols)
                for c in range(0, 600, 7)]
        assert all(a <= b for a, b in zip(long, long[1:]))
        small = [size(n, min(r, rows), cols) if cols >= rows else size(n, rows, min(r, cols))
                 for r in range(1, 129)]
        assert all(a <= b for a, b in zip(small, small[1:]))
