"""The oracle of sequences and log-probabilities against closed forms and independent statements (CPU)."""
import math

import numpy as np
import pytest

from oracle import gdn_oracle as O
from oracle import seq_oracle as Q


@pytest.mark.parametrize("n", [1, 2, 7, 64])
@pytest.mark.parametrize("case", ["plain", "forget", "same_key", "no_update"])
def test_the_chunked_form_is_the_rule(n, case):
    rng = np.random.default_rng(n)
    dk, dv = 8, 5
    q, k = (O.l2_normalise(rng.standard_normal((n, dk)), 1e-6) for _ in range(2))
    v, beta, log_g = rng.standard_normal((n, dv)), rng.random(n), -rng.random(n)
    if case == "forget":
        log_g[n // 2] = -np.inf
    elif case == "same_key":
        k[:], beta[:], log_g[:] = k[0], 1.0, 0.0
    elif case == "no_update":
        beta[:] = 0.0
    T = rng.standard_normal((dk, dv))
    want, S = [], T
    for t in range(n):
        S = np.exp(log_g[t]) * S
        S = S + np.outer(k[t], beta[t] * (v[t] - S.T @ k[t]))
        want.append(S.T @ q[t])
    o, T2 = Q.chunk_step(T, q, k, v, beta, log_g)
    np.testing.assert_allclose(o, want, rtol=0, atol=1e-12 * n)
    np.testing.assert_allclose(T2, S, rtol=0, atol=1e-12 * n)


def test_a_batch_is_its_requests_and_a_sequence_its_parts():
    rng = np.random.default_rng(3)
    d = O.Dims(1, 2, 4, 3, 3)
    lens = [5, 0, 2]
    T, W = rng.standard_normal((3, 2, 4, 3)), rng.standard_normal((3, 2, d.C))
    x, beta, log_g, w = rng.standard_normal((7, d.C)), rng.random((7, 2)), -rng.random((7, 2)), rng.standard_normal((d.C, 3))
    o, T2, W2 = Q.run_batch(lens, T, W, x, beta, log_g, w, d)
    assert np.array_equal(T2[1], T[1]) and np.array_equal(W2[1], W[1])
    first, Ta, Wa = Q.run_sequence(T[0], W[0], x[:2], beta[:2], log_g[:2], w, d)
    rest, Tb, Wb = Q.run_sequence(Ta, Wa, x[2:5], beta[2:5], log_g[2:5], w, d)
    assert np.array_equal(np.concatenate([first, rest]), o[:5]) and np.array_equal(Tb, T2[0]) and np.array_equal(Wb, W2[0])
    assert np.array_equal(W2[0], x[3:5]) and np.array_equal(W2[2], x[5:7])


def test_log_probabilities():
    uniform = np.zeros(8)
    assert np.allclose(Q.log_probabilities(uniform), -math.log(8)) and math.isclose(Q.entropy(uniform), math.log(8))
    row = np.array([1.0, -np.inf, 3.0, 3.0, -2.0])
    p = np.exp(Q.log_probabilities(row))
    assert math.isclose(p.sum(), 1.0) and p[1] == 0.0 and math.isclose(p[2] / p[0], math.exp(2.0))
    assert Q.best_tokens(row, 5) == [2, 3, 0, 4, 1]
    sure = np.array([0.0, 800.0])
    assert Q.entropy(sure) == 0.0 and Q.log_probabilities(sure)[1] == 0.0
