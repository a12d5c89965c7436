"""Pins for the oracle's many-adapter linear and token log probabilities."""

import numpy as np
import pytest

from oracle import adapters, logprobs, lora


def _inputs(seed, d=6, k=5, M=9, n=3, r=2):
    rng = np.random.default_rng(seed)
    f = rng.standard_normal
    return (f((d, k)), f((M, k)), f((n, r, k)), f((n, d, r)), rng.uniform(0.5, 2, n),
            rng.integers(-1, n + 1, M), f((M, d)))


def test_each_token_is_the_single_adapter_layer():
    W, X, A, B, s, ids, _ = _inputs(0)
    Y, H = adapters.forward(W, X, A, B, s, ids)
    for m, a in enumerate(ids):
        if 0 <= a < 3:
            y, h = lora.forward(W, X[m:m + 1], A[a], B[a], s[a])
            assert np.allclose(Y[m], y[0]) and np.allclose(H[m], h[0])
        else:
            assert np.allclose(Y[m], W @ X[m]) and not H[m].any()


def test_adapter_gradients_match_central_differences():
    W, X, A, B, s, ids, dY = _inputs(1)
    dX, dA, dB = adapters.backward(W, X, A, B, s, ids, dY)
    for T, D in ((X, dX), (A, dA), (B, dB)):
        for i in range(0, T.size, 3):
            x0 = T.flat[i]
            v = []
            for e in (1e-5, -1e-5):
                T.flat[i] = x0 + e
                v.append((adapters.forward(W, X, A, B, s, ids)[0] * dY).sum())
            T.flat[i] = x0
            assert abs((v[0] - v[1]) / 2e-5 - D.flat[i]) < 1e-7


def test_logprobs_match_the_definition():
    x = np.log(np.array([[0.1, 0.2, 0.7], [0.5, 0.25, 0.25]])) + 3.0
    lp, ent, tl, ti = logprobs.forward(x, np.array([2, 5]), 2)
    assert np.allclose(lp, [np.log(0.7), 0.0])
    assert np.allclose(ent, [-(0.1 * np.log(0.1) + 0.2 * np.log(0.2) + 0.7 * np.log(0.7)),
                             1.5 * np.log(2)])
    assert ti.tolist() == [[2, 1], [0, 1]] and np.allclose(np.exp(tl), [[0.7, 0.2], [0.5, 0.25]])


def test_logprob_gradient_matches_central_differences():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((4, 7))
    x[1, 2] = -np.inf
    t, g, e = np.array([0, 6, -100, 3]), rng.standard_normal(4), rng.standard_normal(4)
    dx = logprobs.backward(x, t, g, e)
    for i in range(4):
        for j in range(7):
            if np.isinf(x[i, j]):
                assert dx[i, j] == 0
                continue
            v = []
            for h in (1e-5, -1e-5):
                y = x.copy()
                y[i, j] += h
                lp, ent, _, _ = logprobs.forward(y, t)
                v.append((g * lp + e * ent).sum())
            assert abs((v[0] - v[1]) / 2e-5 - dx[i, j]) < 1e-8


@pytest.mark.parametrize("special", [-np.inf, np.inf, np.nan])
def test_special_rows(special):
    x = np.full((1, 4), -np.inf)
    x[0, 1] = special
    lp, ent, tl, ti = logprobs.forward(x, np.array([2]), 2)
    if special == -np.inf:
        assert lp[0] == -np.inf and ent[0] == 0 and ti.tolist() == [[0, 1]]
        assert not logprobs.backward(x, np.array([2]), np.ones(1), np.ones(1)).any()
    else:
        assert np.isnan(lp[0]) and np.isnan(ent[0]) and ti.tolist() == [[1, 0]]
