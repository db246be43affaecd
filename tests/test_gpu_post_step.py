"""The post-training operators together: a step of examples/post_training.py against a float64
evaluation of the same chain.

The step rounds where it says it does (y to bf16, y and the gradient of the logits to e4m3 with
their scales), so the chain is compared link by link, each link's float64 value computed from
what the GPU handed to it; the links' own tolerances are those of their own tests.  For the
whole chain e4m3 (3 mantissa bits, a relative error of 2^-4 at most, about 2^-5 rms, each way)
leaves the gradient's direction: cosine to the unquantised float64 gradient above 0.99.
"""
import importlib.util
import os

import numpy as np
import pytest

from oracle import post_oracle as O
from tests import gpu_harness as H

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("post_training", os.path.join(ROOT, "examples", "post_training.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _cos(a, b):
    a, b = a.ravel(), b.ravel()
    return float(a @ b / np.sqrt((a @ a) * (b @ b)))


def _layernorm_back(dy, x, gamma, eps):
    """dx, dgamma, dbeta in float64, written from the forward formula."""
    mu = x.mean(1, keepdims=True)
    r = 1 / np.sqrt(((x - mu) ** 2).mean(1, keepdims=True) + eps)
    xh = (x - mu) * r
    t = dy * gamma
    return (r * (t - t.mean(1, keepdims=True) - xh * (t * xh).mean(1, keepdims=True)), (dy * xh).sum(0), dy.sum(0))


def _setup(n, hs, V, seed):
    torch = H.torch_cuda()
    ex = _example()
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = (torch.randn(V, hs, device="cuda", generator=g) * hs ** -0.5).to(torch.bfloat16)
    x = torch.randn(n, hs, device="cuda", generator=g).to(torch.bfloat16)
    gamma = 1 + 0.1 * torch.randn(hs, device="cuda", generator=g)
    beta = 0.1 * torch.randn(hs, device="cuda", generator=g)
    return torch, ex, g, w, x, gamma, beta, ex.Step(ex.Head(w), n)


def _whole(x, gamma, beta, w, eps=1e-5):
    """The unquantised chain's logits in float64."""
    y, _, _ = O.layernorm(_f64(x), _f64(gamma), _f64(beta), eps)
    return y @ _f64(w).T


def _chain(dlogits, x, gamma, w, eps=1e-5):
    return _layernorm_back(dlogits @ _f64(w), _f64(x), _f64(gamma), eps)


@pytest.mark.parametrize("n,hs,V", [(1, 64, 160), (37, 256, 1008), (160, 512, 2080)])
def test_policy_step(n, hs, V):
    torch, ex, g, w, x, gamma, beta, step = _setup(n, hs, V, n)
    act = torch.randint(0, V, (n,), device="cuda", generator=g, dtype=torch.int32)
    s0 = _whole(x, gamma, beta, w)
    lp = np.array([O.row_logp(s0[t], int(act[t]))[0] for t in range(n)])
    # ratios of 0.65 and 1: e4m3's error of about 0.04 in a log-probability stays clear of the clip's
    # edges at 0.8 and 1.2, where the gradient jumps
    old = torch.from_numpy(np.float32(lp - np.where(np.arange(n) % 2, np.log(0.65), 0.0))).cuda()
    ref = torch.from_numpy(np.float32(lp + 0.2)).cuda()
    adv = torch.where(torch.arange(n, device="cuda") % 3 == 0, 1.0, -0.5)
    weight = (torch.arange(n, device="cuda") % 5 != 4).float() / n
    dx, dgamma, dbeta = step.policy(x, gamma, beta, act, old, ref, adv, weight)
    torch.cuda.synchronize()
    # link: the product of what was quantised
    q, s = (H.host(t) for t in (step.yq, step.ys))
    wq, ws = O.quant_rows(step.y.float().cpu().numpy())
    assert np.array_equal(q, wq) and np.array_equal(s, ws)
    # link: the gradient handed back, and the norm's backward pass over it
    want = _layernorm_back(_f64(step.dy), _f64(x), _f64(gamma), 1e-5)
    assert np.abs(_f64(dx) - want[0]).max() <= 2.0 ** -8 * np.abs(want[0]).max() + 1e-6 * np.abs(_f64(step.dy)).max()
    for got, ref64 in ((dgamma, want[1]), (dbeta, want[2])):
        assert np.abs(_f64(got) - ref64).max() <= 1e-5 * np.abs(_f64(step.dy)).sum(0).max() * 4
    # the whole chain
    ol = O.policy(s0, act.cpu().numpy(), _f64(old), _f64(ref), _f64(adv), _f64(weight), 0.2, 0.2, 0.04, 1.0)
    full = _chain(ol["grad"], x, gamma, w)
    for got, ref64 in zip((dx, dgamma, dbeta), full):
        assert _cos(_f64(got), ref64) > 0.99
    # rows that do not count get no gradient; what is left of the logits is theirs alone
    dead = _f64(weight) == 0
    assert not _f64(step.dx)[dead].any() and not _f64(step.logits)[dead].any()


def test_preference_step():
    pairs, length, hs, V = 3, 10, 256, 1040
    n = 2 * pairs * length
    torch, ex, g, w, x, gamma, beta, step = _setup(n, hs, V, 5)
    labels = torch.randint(0, V, (n,), device="cuda", generator=g, dtype=torch.int32)
    weight = (torch.arange(n, device="cuda") % length >= 3).float()
    start = torch.arange(2 * pairs + 1, device="cuda", dtype=torch.int64) * length
    ref = -50 + torch.randn(2 * pairs, device="cuda", generator=g)
    loss, margin, pi = (torch.empty(k, device="cuda") for k in (pairs, pairs, 2 * pairs))
    grads = step.preference(x, gamma, beta, labels, weight, start, pairs, ref, loss, margin, pi)
    torch.cuda.synchronize()
    o = O.preference(_whole(x, gamma, beta, w), labels.cpu().numpy(), _f64(weight), start.cpu().numpy(), pairs, _f64(ref),
                     0.1, 0.0, 0, 1.0 / pairs)
    for got, want in zip(grads, _chain(o["grad"], x, gamma, w)):
        assert _cos(_f64(got), want) > 0.99


def test_step_in_a_graph():
    """A captured step gives the eager step's bits (no allocation and no host read in it)."""
    n, hs, V = 64, 256, 1024
    torch, ex, g, w, x, gamma, beta, step = _setup(n, hs, V, 9)
    act = torch.randint(0, V, (n,), device="cuda", generator=g, dtype=torch.int32)
    old = torch.full((n,), -7.0, device="cuda")
    adv = torch.randn(n, device="cuda", generator=g)
    weight = torch.full((n,), 1.0 / n, device="cuda")
    eager = [t.clone() for t in step.policy(x, gamma, beta, act, old, old, adv, weight)]
    total = step.total.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.policy(x, gamma, beta, act, old, old, adv, weight)
    for t in (step.dx, step.dgamma, step.dbeta, step.total):
        t.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(eager + [total], (step.dx, step.dgamma, step.dbeta, step.total)):
        assert torch.equal(a, b)


def test_training_improves():
    ex = _example()
    H.torch_cuda()
    was, now = ex.train_policy(128, 256, 256, 30)
    assert now > was + 0.05
    first, last = ex.train_preference(4, 16, 256, 1024, 8)
    assert last[0] < first[0] and last[1] > first[1]
