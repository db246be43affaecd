"""How exactly the preference loss keeps the sums over a sequence, and values at the ends of their ranges.

A row of two columns whose other logit c is 200 or more has the log-probability -c exactly (the
picked column's exponential is below the smallest float, so m = c, ln S = 0), so that sums over
such rows are known to the last bit from the inputs alone.
"""
from fractions import Fraction

import numpy as np
import pytest

from tests.test_gpu_post_loss import run_policy, run_pref

pytestmark = pytest.mark.gpu
INF = float("inf")


def _exact_rows(c):
    """Logits of rows whose label 0 has log-probability -c."""
    return np.stack([np.zeros_like(c), c], 1).astype(np.float32)


def _sum(w, c):
    return sum((-Fraction(float(a)) * Fraction(float(b)) for a, b in zip(w, c)), Fraction(0))


def test_sequence_sums_keep_48_bits():
    """Terms of some 1000 that cancel to less than 0.1: each term's rounding to fp32 would be
    far larger than what is allowed here, 2^-24 of the sum and 2^-40 of its terms' sizes."""
    g = np.random.default_rng(5)
    n = 600
    c = g.uniform(200, 2000, n).astype(np.float32)
    w = g.uniform(0.3, 1.7, n).astype(np.float32)
    c[1::2], w[1::2] = c[::2], -w[::2] * np.float32(1 - 1e-4)
    half = n // 2
    got = run_pref(_exact_rows(c), np.zeros(n, np.uint32), w, [0, half, n], 1, None, 0.125, 0.0, 1, 1.0, "f32")
    for s, sl in enumerate((slice(0, half), slice(half, n))):
        want, size = _sum(w[sl], c[sl]), float(np.abs(w[sl].astype(np.float64) * c[sl]).sum())
        assert abs(Fraction(float(got["seq"][s])) - want) <= Fraction(2.0 ** -24) * abs(want) + Fraction(2.0 ** -40 * size)


@pytest.mark.parametrize("n", [40, 129, 700])
def test_margin_of_long_sequences(n):
    """Sums of some -200 n less references of the same size: the margin is that of the inputs to a
    few roundings of itself (the products with beta and the last sum: 4 * 2^-24) and 2^-40 of the sums."""
    g = np.random.default_rng(n)
    pairs = 4
    c = g.uniform(200, 260, 2 * pairs * n).astype(np.float32)
    w = np.where(np.arange(c.size) % n < n // 8, 0, g.uniform(0.5, 1.5, c.size)).astype(np.float32)
    start = np.arange(2 * pairs + 1) * n
    pi = [_sum(w[a:b], c[a:b]) for a, b in zip(start, start[1:])]
    ref = np.array([float(p) for p in pi]) + 3 * g.normal(size=2 * pairs)
    ref = ref.astype(np.float32)
    beta = np.float32(0.1)
    got = run_pref(_exact_rows(c), np.zeros(c.size, np.uint32), w, start, pairs, ref, float(beta), 0.1, 0, 1.0, "f32")
    for i in range(pairs):
        want = Fraction(float(beta)) * ((pi[i] - Fraction(float(ref[i]))) - (pi[pairs + i] - Fraction(float(ref[pairs + i]))))
        tol = Fraction(4 * 2.0 ** -24) * abs(want) + Fraction(float(beta) * 2.0 ** -40) * (abs(pi[i]) + abs(pi[pairs + i]))
        assert abs(Fraction(float(got["margin"][i])) - want) <= tol, (i, float(want), got["margin"][i])


@pytest.mark.parametrize("V", [40, 3000, 9000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_preference_of_impossible_labels(V, dtype):
    """A label of probability 0 (logit -inf) in the rejected sequence: the pair is won beyond doubt,
    loss 0, nothing to learn; in the chosen one the loss is infinite and the gradient is beta's."""
    g = np.random.default_rng(V)
    x = (g.integers(-8, 9, (8, V)) * 0.5).astype(np.float32)
    lab = g.integers(0, V, 8).astype(np.uint32)
    start = [0, 2, 4, 6, 8]                                  # pairs (0, 2) and (1, 3) of sequences of two rows
    x[[2, 3, 6, 7], lab[[2, 3, 6, 7]]] = 0.0                 # pair 1 is close
    x[5, lab[5]] = -np.inf                                   # sequence 2: rejected in pair 0
    w = np.ones(8, np.float32)
    for kind, won in ((0, 0.0), (2, 0.0)):
        got = run_pref(x, lab, w, start, 2, None, 0.5, 0.0, kind, 1.0, dtype)
        assert got["margin"][0] == INF and got["seq"][2] == -INF and got["loss"][0] == won, (kind, got["loss"])
        assert np.isfinite(got["loss"][1]) and got["mean"] == pytest.approx(got["loss"][1] / 2, rel=1e-6)
        assert not got["grad"][[0, 1, 4, 5]].any() and got["grad"][[2, 3, 6, 7]].any()
    got = run_pref(x, lab, w, start, 2, None, 0.5, 0.1, 0, 1.0, dtype)        # smoothed: the doubt costs without end
    assert got["loss"][0] == INF
    x[5, lab[5]], x[0, lab[0]] = 1.0, -np.inf                # now the chosen one
    got = run_pref(x, lab, w, start, 2, None, 0.5, 0.0, 0, 1.0, dtype)
    assert got["margin"][0] == -INF and got["loss"][0] == INF and np.isfinite(got["grad"]).all()
    assert got["grad"][0, lab[0]] == -0.5                    # beta ([j == a] - 0), a step up
    # impossible on both sides: no answer
    x[5, lab[5]] = -np.inf
    assert np.isnan(run_pref(x, lab, w, start, 2, None, 0.5, 0.0, 0, 1.0, dtype)["loss"][0])


@pytest.mark.parametrize("V", [40, 3000, 9000])
@pytest.mark.parametrize("hi", [0.28, INF])
def test_policy_of_no_advantage(V, hi):
    """An advantage of 0 costs nothing and teaches nothing, however far the ratio has gone (here past
    the largest float: the sampler's log-probability was below -89, or it was -inf)."""
    g = np.random.default_rng(V)
    n = 6
    x = (g.normal(size=(n, V)) * 2).astype(np.float32)
    act = g.integers(0, V, n).astype(np.uint32)
    old = np.array([-120.0, -np.inf, -8.0, -150.0, -1e30, -8.0], np.float32)
    adv = np.array([0.0, -0.0, 0.0, 0.0, 0.0, 1.0], np.float32)
    w = np.ones(n, np.float32)
    got = run_policy(x, act, old, None, adv, w, 0.0, 1.0, "f32", hi=hi)
    assert not got["loss"][:5].any() and not got["grad"][:5].any() and np.isfinite(got["total"]), got["loss"]
    # beside a KL term that is all there is
    ref = np.full(n, -9.0, np.float32)
    a = run_policy(x, act, old, ref, adv, w, 0.5, 1.0, "f32", hi=hi)
    b = run_policy(x, act, np.full(n, -8.0, np.float32), ref, np.where(adv == 0, 0, adv).astype(np.float32), w, 0.5, 1.0, "f32", hi=hi)
    assert np.isfinite(a["loss"]).all() and np.array_equal(a["loss"], b["loss"]) and np.array_equal(a["grad"], b["grad"])
    # with an advantage the vast ratio counts: clipped on the side that gains, without bound on the other
    adv = np.array([1.0, 1.0, 1.0, -1.0, -2.0, 1.0], np.float32)
    got = run_policy(x, act, old, None, adv, w, 0.0, 1.0, "f32", hi=0.28)
    assert np.allclose(got["loss"][:2], -1.28, rtol=1e-6) and got["loss"][3] == INF and got["loss"][4] == INF
    # NaN stays NaN
    x[0, 1] = np.nan
    assert np.isnan(run_policy(x, act, old, None, adv * 0, w, 0.0, 1.0, "f32", hi=hi)["loss"][0])
