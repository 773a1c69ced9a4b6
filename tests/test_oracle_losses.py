"""Pins of the float64 row losses: closed forms on two-token rows, differences of the loss against the
gradient, and the rules for rows that do not count."""
import math

import numpy as np
import pytest

from oracle import losses


def _diff(f, x, h=1e-6):
    """Central differences of f at every entry of x."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


def test_policy_two_tokens_closed_form():
    # p(0) = s(a - b); without clipping the loss is -p(0) A / q
    a, b, q, A = 0.3, -0.4, 0.6, 1.7
    s = 1 / (1 + math.exp(b - a))
    r = losses.policy_loss([[a, b]], [0], [math.log(q)], [A], clip_low=10, clip_high=10)
    assert r["row_loss"][0] == pytest.approx(-s * A / q, rel=1e-14)
    # d/da of -A s(a - b) / q is -A s (1 - s) / q
    assert r["grad"][0] == pytest.approx([-A * s * (1 - s) / q, A * s * (1 - s) / q], rel=1e-13)
    assert r["entropy"][0] == pytest.approx(-s * math.log(s) - (1 - s) * math.log(1 - s), rel=1e-13)


@pytest.mark.parametrize("A,ratio,clipped", [(1.0, 1.5, True), (1.0, 0.5, False), (-1.0, 0.5, True),
                                             (-1.0, 1.5, False), (1.0, 1.1, False), (-1.0, 0.9, False)])
def test_policy_clipping(A, ratio, clipped):
    x = np.array([[0.2, 0.1, -0.5]])
    lp = x[0, 1] - math.log(np.exp(x).sum())
    r = losses.policy_loss(x, [1], [lp - math.log(ratio)], [A], clip_low=0.2, clip_high=0.3)
    want = min(ratio * A, min(max(ratio, 0.8), 1.3) * A)
    assert r["loss"] == pytest.approx(-want, rel=1e-12)
    assert np.all(r["grad"] == 0) == clipped


@pytest.mark.parametrize("ent,kl,T", [(0.0, 0.0, 1.0), (0.05, 0.0, 0.7), (0.0, 0.3, 1.4), (0.1, 0.2, 0.6)])
def test_policy_gradient_against_differences(ent, kl, T):
    rng = np.random.default_rng(5)
    B, V = 5, 9
    x = rng.standard_normal((B, V)) * 2
    tok = rng.integers(0, V, B)
    allowed = rng.random((B, V)) < 0.7
    allowed[np.arange(B), tok] = True
    adv = rng.standard_normal(B)
    w = np.array([0.3, 0.0, 0.5, 1.0, 0.2])

    def call(y):
        base = losses.policy_loss(x, tok, np.zeros(B), adv, weight=w, T=T, allowed=allowed)["logprob"]
        return losses.policy_loss(y, tok, base + [0.05, 0, -0.4, 0.4, 0.1], adv, base - 0.2, w, kl=kl, ent=ent,
                                  T=T, allowed=allowed)

    assert np.allclose(call(x)["grad"], _diff(lambda y: call(y)["loss"], x), atol=2e-9)


def test_policy_rows_that_do_not_count():
    x = np.array([[1.0, 2.0], [np.nan, np.nan], [3.0, 1.0], [0.5, 0.25]])
    allowed = np.array([[True, True], [True, True], [False, True], [False, False]])
    r = losses.policy_loss(x, [-1, 0, 0, 0], np.zeros(4), np.ones(4), weight=[1, 0, 1, 1], ent=0.1, allowed=allowed)
    assert r["loss"] == 0 and np.all(r["grad"] == 0) and np.all(r["row_loss"] == 0)
    assert r["logprob"][0] == 0 and r["logprob"][1] == 0
    assert r["logprob"][2] == -np.inf and np.isnan(r["logprob"][3])


def test_preference_closed_form():
    # one-token answers of two-token rows: R is ln s(a - b)
    x = np.array([[0.4, -0.3], [0.1, 0.9]])
    r = losses.preference_loss(x, [0, 1], [0, 1, 2], beta=0.5)
    lp = [-math.log1p(math.exp(-0.7)), -math.log1p(math.exp(-0.8))]
    h = 0.5 * (lp[0] - lp[1])
    assert r["loss"] == pytest.approx(math.log1p(math.exp(-h)), rel=1e-14)
    assert r["reward"] == pytest.approx([0.5 * v for v in lp], rel=1e-13)


@pytest.mark.parametrize("smooth,margin,average,T", [(0.0, 0.0, False, 1.0), (0.2, 0.0, False, 0.8),
                                                     (0.0, 0.6, True, 1.0), (0.1, -0.3, True, 1.7)])
def test_preference_gradient_against_differences(smooth, margin, average, T):
    rng = np.random.default_rng(6)
    start = [0, 3, 3, 5, 9]  # an empty sequence among them
    N, V = 9, 6
    x = rng.standard_normal((N, V))
    tok = rng.integers(0, V, N)
    tok[4] = -1
    w = rng.choice([0.0, 1.0, 0.5], N)
    ref = rng.standard_normal(N) - 2

    def call(y):
        return losses.preference_loss(y, tok, start, w, ref, 0.7, smooth, margin, average, T)

    assert np.allclose(call(x)["grad"], _diff(lambda y: call(y)["loss"], x), atol=2e-9)
