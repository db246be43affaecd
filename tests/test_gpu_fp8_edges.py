"""The quantisers' zeros, vocabularies that are no multiple of 16 on the way back, and few-row products of
more tiles than CTAs.  Tolerances as in test_gpu_fp8.py."""
import numpy as np
import pytest

from oracle import post_oracle as O
from tests import gpu_harness as H
from tests.test_gpu_fp8 import _bf, _data, product

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [128, 130, 257])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantise_keeps_the_sign_of_zero(K, dtype):
    """x / scale of -0 is -0, whichever way the quotient is taken (a block of zeros divides)."""
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    M = 9
    x = _data(M, K, K)
    x[:, ::3], x[:, 1::5] = -0.0, 0.0
    x[:, 2::7] *= np.float32(1e-30)                          # to +0 and -0 in e4m3
    x[4] = -0.0
    if dtype == "bf16":
        x = _bf(x).float().numpy()
    t = torch.from_numpy(x).cuda()
    q = torch.empty(M, K, dtype=torch.uint8, device="cuda")
    s = torch.empty(-(-K // 128), M, device="cuda")
    if dtype == "bf16":
        vl.vl_quant_fp8_rows_bf16(t.to(torch.bfloat16), K, M, K, q, s)
    else:
        vl.vl_quant_fp8_rows(t, K, M, K, q, s)
    wq, ws = O.quant_rows(x)
    assert np.array_equal(H.host(s), ws) and np.array_equal(H.host(q), wq)
    if dtype == "bf16":
        s = torch.empty(1, -(-K // 128), device="cuda")
        vl.vl_quant_fp8_blocks_bf16(t.to(torch.bfloat16), M, K, q, s)
        wq, ws = O.quant_blocks(x)
        assert np.array_equal(H.host(s), ws) and np.array_equal(H.host(q), wq)


@pytest.mark.parametrize("M", [5, 64, 70])
def test_way_back_of_a_vocabulary_no_multiple_of_16(M):
    """V = 1003: gradient rows of stride 1008 whose last columns are zero, and a transposed plane padded
    the same way, give dx; the columns of padding add nothing."""
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    V, pad, hs = 1003, 1008, 256
    g = np.random.default_rng(M)
    w = _bf(g.normal(size=(V, hs))).float().numpy()
    logits = torch.zeros(M, pad, device="cuda")              # the padding is zeroed once and never written
    logits[:, :V] = torch.from_numpy(g.normal(size=(M, V)).astype(np.float32)).cuda()
    act = torch.randint(0, V, (M,), device="cuda", dtype=torch.int32)
    old, adv, wt = (torch.full((M,), v, device="cuda") for v in (-7.0, 1.0, 1.0))
    loss = torch.empty(M, device="cuda")
    vl.vl_policy_loss(logits, pad, M, V, act, old, None, adv, wt, 0.2, 1.0, 0.0, 1.0, logits, pad, loss)
    torch.cuda.synchronize()
    grad = H.host(logits)
    assert not grad[:, V:].any() and grad[:, :V].any()
    back = np.zeros((hs, pad), np.float32)
    back[:, :V] = w.T
    bq, bs = torch.empty(hs, pad, dtype=torch.uint8, device="cuda"), torch.empty(2, 8, device="cuda")
    vl.vl_quant_fp8_blocks_bf16(_bf(back).cuda(), hs, pad, bq, bs)
    gq, gs = torch.empty(M, pad, dtype=torch.uint8, device="cuda"), torch.empty(8, M, device="cuda")
    vl.vl_quant_fp8_rows(logits, pad, M, pad, gq, gs)
    dx = torch.empty(M, hs, device="cuda")
    vl.vl_gemm_fp8_tn(gq, gs, bq, bs, dx, M, hs, pad, hs)
    qa, sa = O.quant_rows(np.pad(grad[:, :V], ((0, 0), (0, pad - V))))
    qb, sb = O.quant_blocks(back)
    assert np.array_equal(H.host(gq), qa) and np.array_equal(H.host(bq), qb)
    # the sums over V columns alone
    want, mag = O.gemm_fp8(qa[:, :V], sa, qb[:, :V], sb)
    assert (np.abs(H.host(dx) - want) <= (2 * 128 + 8 + 8) * H.EPS * mag).all()


@pytest.mark.parametrize("M", [3, 20, 50])
def test_product_of_few_rows_and_many_tiles(M):
    """More 128-row tiles of the plane than two CTAs an SM take at once, and more than one batch of scales."""
    product(M, 40001, 1040)


def test_step_of_a_vocabulary_no_multiple_of_16():
    """The example's steps at V = 1003: the gradients keep the direction of the unquantised ones (cosine above 0.99, as
    at multiples of 16), and the padding stays zero."""
    from tests.test_gpu_post_step import _chain, _cos, _f64, _setup, _whole

    n, hs, V = 60, 256, 1003
    torch, ex, g, w, x, gamma, beta, step = _setup(n, hs, V, 3)
    act = torch.randint(0, V, (n,), device="cuda", generator=g, dtype=torch.int32)
    s0 = _whole(x, gamma, beta, w)
    # ratios of 1: e4m3's error of about 0.04 in a log-probability stays clear of the clip's edges
    old = torch.from_numpy(np.float32([O.row_logp(s0[t], int(act[t]))[0] for t in range(n)])).cuda()
    adv, weight = torch.where(torch.arange(n, device="cuda") % 3 == 0, 1.0, -0.5), torch.full((n,), 1 / n, device="cuda")
    grads = step.policy(x, gamma, beta, act, old, None, adv, weight)
    o = O.policy(s0, act.cpu().numpy(), _f64(old), None, _f64(adv), _f64(weight), 0.2, 0.2, 0.0, 1.0)
    for got, want in zip(grads, _chain(o["grad"], x, gamma, w)):
        assert _cos(_f64(got), want) > 0.99
    base = step.logits._base if step.logits._base is not None else step.logits
    assert tuple(base.shape) == (n, 1008) and not bool(base[:, V:].any())
    start = torch.arange(5, device="cuda", dtype=torch.int64) * (n // 4)
    loss, margin, pi = (torch.empty(k, device="cuda") for k in (2, 2, 4))
    grads = step.preference(x, gamma, beta, act, weight * n, start, 2, None, loss, margin, pi)
    o = O.preference(s0, act.cpu().numpy(), np.ones(n), start.cpu().numpy(), 2, None, 0.1, 0.0, 0, 0.5)
    for got, want in zip(grads, _chain(o["grad"], x, gamma, w)):
        assert _cos(_f64(got), want) > 0.99
    assert not bool(base[:, V:].any())
