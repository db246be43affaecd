"""The 8-bit head product and its quantisers on the GPU against float64.

The quantisers are bit-exact (an fp32 product, an fp32 division and one rounding).  The product: e4m3 products
are exact in fp32; a block's 128 of them are summed in fp32 (any order, each step off by at most
2^-23 of the running size), then scaled and added over the blocks, so
|d| <= (2 * 128 + ceil(K / 128) + 8) * 2^-24 * sum |a b|.
"""
import numpy as np
import pytest

from oracle import post_oracle as O
from tests import gpu_harness as H

pytestmark = pytest.mark.gpu


def _bf(a):
    torch = H.torch_cuda()
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16)


def _data(M, K, seed):
    g = np.random.default_rng(seed)
    x = g.normal(size=(M, K)) * np.exp(g.normal(size=(M, 1)))
    x[:, g.integers(0, K, max(1, K // 100))] *= 30
    return x.astype(np.float32)


@pytest.mark.parametrize("M,K,pad", [(1, 16, 0), (3, 128, 0), (5, 130, 1), (17, 272, 8), (130, 4096, 0), (9, 1000, 3), (2, 1, 0)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantise_rows(M, K, pad, dtype):
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    x = _data(M, K, M + K)
    x[0, :min(K, 128)] = 0                                  # an empty block
    if M > 2:
        x[1, 0], x[2, K - 1] = 1e-38, 3e38                  # near the ends of the range
    if dtype == "bf16":
        x = _bf(x).float().numpy()
    buf = torch.full((M, K + pad), 5.0, device="cuda")
    buf[:, :K] = torch.from_numpy(x).cuda()
    if dtype == "bf16":
        buf = buf.to(torch.bfloat16)
    kb = -(-K // 128)
    q = torch.full((M * K + 16,), 0xAA, dtype=torch.uint8, device="cuda")
    s = torch.full((kb * M + 4,), 9.0, device="cuda")
    (vl.vl_quant_fp8_rows_bf16 if dtype == "bf16" else vl.vl_quant_fp8_rows)(buf, K + pad, M, K, q, s)
    torch.cuda.synchronize()
    wq, ws = O.quant_rows(x)
    assert np.array_equal(H.host(s)[:kb * M].reshape(kb, M), ws) and (H.host(s)[kb * M:] == 9).all()
    assert np.array_equal(H.host(q)[:M * K].reshape(M, K), wq) and (H.host(q)[M * K:] == 0xAA).all()


@pytest.mark.parametrize("scales", ["any", "round", "small", "large"])
def test_quantise_near_the_middles(scales):
    """Values a few ulps around the middles between e4m3 values, over scales of every kind (round
    ones: within 9 ulps of a short number): the bytes are those of an fp32 division."""
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    M = 6000
    g = np.random.default_rng(len(scales))
    amax = np.float32(448) * np.exp(g.uniform(-20, 20, M)).astype(np.float32)
    if scales == "round":
        amax = (np.float32(448) * g.integers(8, 16, M).astype(np.float32) * np.exp2(g.integers(-20, 20, M)).astype(np.float32))
    elif scales == "small":
        amax = np.exp2(g.uniform(-126, -60, M)).astype(np.float32)
    elif scales == "large":
        amax = np.exp2(g.uniform(100, 127.9, M)).astype(np.float32)
    amax = (amax.view(np.int32) + g.integers(-9, 10, M).astype(np.int32)).view(np.float32)
    s = np.maximum(amax, np.float32(2.0 ** -100)) * (np.float32(1) / np.float32(448))
    v = np.sort(np.abs(O.e4m3_value(np.arange(0x7F))))
    mid = ((v[1:] + v[:-1]) / 2).astype(np.float32)
    x = mid[g.integers(0, len(mid), (M, 128))] * s[:, None]
    x = (x.view(np.int32) + g.integers(-3, 4, x.shape).astype(np.int32)).view(np.float32)
    x = np.minimum(np.abs(x), amax[:, None]) * g.choice(np.float32([-1, 1]), x.shape)
    x[:, 0] = amax
    q = torch.empty(M, 128, dtype=torch.uint8, device="cuda")
    sa = torch.empty(1, M, device="cuda")
    vl.vl_quant_fp8_rows(torch.from_numpy(x).cuda(), 128, M, 128, q, sa)
    wq, ws = O.quant_rows(x)
    assert np.array_equal(H.host(sa), ws) and np.array_equal(H.host(q), wq)


@pytest.mark.parametrize("N,K", [(1, 16), (128, 128), (129, 130), (300, 1000), (64, 2064)])
def test_quantise_blocks(N, K):
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    w = _bf(_data(N, K, N * K))
    w[:, :8] = 0
    nb, kb = -(-N // 128), -(-K // 128)
    q = torch.full((N * K + 16,), 0xAA, dtype=torch.uint8, device="cuda")
    s = torch.full((nb * kb + 4,), 9.0, device="cuda")
    vl.vl_quant_fp8_blocks_bf16(w.cuda(), N, K, q, s)
    torch.cuda.synchronize()
    wq, ws = O.quant_blocks(w.float().numpy())
    assert np.array_equal(H.host(s)[:nb * kb].reshape(nb, kb), ws) and (H.host(s)[nb * kb:] == 9).all()
    assert np.array_equal(H.host(q)[:N * K].reshape(N, K), wq) and (H.host(q)[N * K:] == 0xAA).all()


def test_quantise_specials():
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    x = _data(4, 256, 3)
    x[1, 5], x[2, 200] = np.nan, np.inf
    q, s = torch.empty(4, 256, dtype=torch.uint8, device="cuda"), torch.empty(2, 4, device="cuda")
    vl.vl_quant_fp8_rows(H.dev(x), 256, 4, 256, q, s)
    torch.cuda.synchronize()
    v, sc = O.e4m3_value(H.host(q)), H.host(s)
    wq, ws = O.quant_rows(x)
    assert np.isnan(v[1, 5]) and np.isnan(v[2, 200]) and np.isinf(sc[1, 2])
    keep = np.ones((4, 256), bool)
    keep[1, 5] = keep[2, 128:] = False
    assert np.array_equal(H.host(q)[keep], wq[keep])


def product(M, N, K, pad=0, off=0, alpha=1.0, seed=0, stream=None):
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    qa, sa = O.quant_rows(_data(M, K, seed + M))
    qb, sb = O.quant_blocks(_data(N, K, seed + N + 1))
    ld = N + pad
    buf = torch.full((off + M * ld + 8,), 5.0, device="cuda")
    D = buf[off:off + M * ld].view(M, ld)
    dev = [H.dev(v) for v in (qa, sa, qb, sb)]
    torch.cuda.synchronize()
    vl.vl_gemm_fp8_tn(*dev, D.data_ptr(), M, N, K, ld, alpha, stream)
    torch.cuda.synchronize()
    got = H.host(buf)
    assert (got[:off] == 5).all() and (got[off + M * ld:] == 5).all()
    got = got[off:off + M * ld].reshape(M, ld)
    assert (got[:, N:] == 5).all()
    want, mag = O.gemm_fp8(qa, sa, qb, sb, float(np.float32(alpha)))
    tol = (2 * 128 + -(-K // 128) + 8) * H.EPS * mag
    err = np.abs(got[:, :N] - want)
    assert (err <= tol).all(), (M, N, K, float((err / np.maximum(tol, 1e-300)).max()), np.argwhere(err > tol)[:4].tolist())
    H.report("fp8 product", "max error / bound", float((err / np.maximum(tol, 1e-300)).max()))


@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 128, 128), (3, 7, 144), (16, 300, 256), (128, 256, 512), (129, 257, 400),
                                   (200, 1000, 1040), (1, 5000, 2048), (130, 513, 4096), (513, 130, 272), (300, 2000, 640)])
def test_product(M, N, K):
    product(M, N, K)


def test_product_strides_alignment_alpha_and_stream():
    torch = H.torch_cuda()
    for pad, off in ((1, 0), (4, 1), (3, 2), (0, 3)):
        product(65, 384, 256, pad=pad, off=off, alpha=-0.37)
    product(40, 700, 384, stream=torch.cuda.Stream())


def test_product_many_tiles_a_cta():
    product(700, 20001, 256)


def test_product_long_contraction():
    """The backward product: few columns, the vocabulary as the contraction."""
    product(40, 256, 32000)
    product(5, 130, 50256)


def test_product_nan_and_zero_scales():
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    qa, sa = O.quant_rows(_data(4, 256, 1))
    qb, sb = O.quant_blocks(_data(130, 256, 2))
    sa[:, 2] = 0
    sa[1, 1] = np.nan
    D = torch.empty(4, 130, device="cuda")
    vl.vl_gemm_fp8_tn(*(H.dev(v) for v in (qa, sa, qb, sb)), D, 4, 130, 256, 130)
    torch.cuda.synchronize()
    d = H.host(D)
    assert np.isnan(d[1]).all() and not d[2].any() and np.isfinite(d[[0, 3]]).all()
