"""The float64 definitions of the post-training operators against facts that do not come from
themselves: hand values, central differences, torch's own float8 rounding."""
import math

import numpy as np
import pytest

from oracle import post_oracle as O


def _fd(f, x, h=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


def test_policy_by_hand():
    # two equal logits: logp = -ln 2, p = 1/2
    x = np.zeros((4, 2))
    old = np.array([-math.log(2)] * 2 + [-math.log(2) - math.log(2)] * 2)     # ratios 1, 1, 2, 2
    adv = np.array([3.0, -3.0, 3.0, -3.0])
    o = O.policy(x, np.zeros(4, int), old, None, adv, np.ones(4), 0.2, 0.25, 0.0, 1.0)
    assert np.allclose(o["loss"], [-3, 3, -3.75, 6])
    assert np.allclose(o["G"], [-3, 3, 0, 6])
    assert np.allclose(o["grad"][1], [1.5, -1.5]) and not o["grad"][2].any()


def test_policy_gradient_against_differences():
    g = np.random.default_rng(5)
    x, act = g.normal(size=(6, 5)), g.integers(0, 5, 6)
    lp = np.array([O.row_logp(x[t], act[t])[0] for t in range(6)])
    old, ref, adv, w = lp - g.normal(size=6) * 0.4, lp + g.normal(size=6), g.normal(size=6), g.random(6)
    w[2] = 0
    args = (act, old, ref, adv, w, 0.2, 0.28, 0.3, 1.7)
    f = lambda y: 1.7 * O.policy(y, *args)["total"]  # noqa: E731
    assert np.allclose(O.policy(x, *args)["grad"], _fd(f, x), atol=1e-8)


@pytest.mark.parametrize("kind", [0, 1, 2])
def test_preference_gradient_against_differences(kind):
    g = np.random.default_rng(kind)
    start = np.array([0, 2, 5, 6, 8])
    x, lab = g.normal(size=(9, 4)), g.integers(0, 4, 9)
    w, ref = g.random(9), g.normal(size=4)
    w[3] = 0
    args = (lab, w, start, 2, ref, 0.3, 0.1, kind, 0.5)
    f = lambda y: 0.5 * O.preference(y, *args)["loss"].sum()  # noqa: E731
    got = O.preference(x, *args)
    assert np.allclose(got["grad"], _fd(f, x), atol=1e-8)
    assert not got["grad"][8].any()          # a row of no sequence


def test_pair_loss_by_hand():
    assert np.allclose(O.pair_loss(0.0, 0.1, 0.0, 0), (math.log(2), -0.05))
    assert np.allclose(O.pair_loss(7.0, 0.1, 0.0, 1), (4.0, 4.0))
    assert O.pair_loss(20.0, 0.1, 0.0, 2) == (0.0, 0.0)
    assert O.pair_loss(5000.0, 1.0, 0.25, 0)[0] == pytest.approx(1250.0)


def test_layernorm_gradient_against_differences():
    g = np.random.default_rng(3)
    x, dy, ga, be = g.normal(size=(3, 7)), g.normal(size=(3, 7)), g.normal(size=7), g.normal(size=7)
    y, mu, rstd = O.layernorm(x, ga, be, 1e-5)
    dx, dg, db = O.layernorm_bwd(dy, x, ga, mu, rstd)
    assert np.allclose(dx, _fd(lambda v: (O.layernorm(v, ga, be, 1e-5)[0] * dy).sum(), x), atol=1e-7)
    assert np.allclose(dg, _fd(lambda v: (O.layernorm(x, v, be, 1e-5)[0] * dy).sum(), ga), atol=1e-7)
    assert np.allclose(db, _fd(lambda v: (O.layernorm(x, ga, v, 1e-5)[0] * dy).sum(), be), atol=1e-7)
    assert np.allclose(y.mean(0) * 3, y.sum(0))


def test_e4m3_matches_torch():
    torch = pytest.importorskip("torch")
    b = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(b).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(O.e4m3_value(b), t, equal_nan=True)
    g = np.random.default_rng(1)
    v = np.concatenate([g.normal(size=4000) * 100, g.normal(size=4000) * 0.01, t[~np.isnan(t)],
                        (t[:126] + t[1:127]) / 2]).astype(np.float32)
    v = v[np.abs(v) <= 448]
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(O.e4m3_byte(v), want)


def test_quantised_product_is_near_the_product():
    g = np.random.default_rng(2)
    a, b = g.normal(size=(5, 272)).astype(np.float32), g.normal(size=(130, 272)).astype(np.float32)
    qa, sa = O.quant_rows(a)
    qb, sb = O.quant_blocks(b)
    y, mag = O.gemm_fp8(qa, sa, qb, sb)
    want = a.astype(np.float64) @ b.astype(np.float64).T
    # each factor is within 2^-4 of itself or half a step of the smallest spacing of its block
    assert np.all(np.abs(y - want) <= 2.2 * 2.0 ** -4 * mag + 1e-3)
