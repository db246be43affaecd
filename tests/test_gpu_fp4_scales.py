"""Row scales of the 4-bit product from one end of fp32 to the other.

Values of e2m1, block scales and row scales are powers of two times small whole numbers here, so that the sum over K is exact
in fp32 and D = alpha ra rb sum is exact too, rounded to D's type (infinite or 0 where it has to be): the comparison is of bits
down to 2^-126.  Below, a product on the way may be subnormal already: it is off by at most 2^-150, the power of two that follows is
1/2 or less (it is 1 where nothing has to be kept in range), and the result rounds once more by 2^-150: 0.75 x 2^-149 in all.  In
bf16 half a subnormal step, 2^-134, comes on top.
"""
import numpy as np
import pytest

from oracle import draft_oracle as O
from tests import gpu_harness as H

pytestmark = pytest.mark.gpu


def product(M, N, K, ea, eb, alpha, bf16, pad=0, blocks=(0x30, 0x38, 0x40)):
    """Checks the product whose rows' scales are 2^ea [M] and 2^eb [N]; blocks: bytes of their blocks' scales, each twice the one
    before."""
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    g = np.random.default_rng(M + K)
    kb = -(-K // 16)

    def rows(m):
        c = (g.integers(1, 8, (m, K)) | 8 * g.integers(0, 2, (m, K))).astype(np.uint8)     # no zeros
        return c, g.choice(np.uint8(blocks), (m, kb))

    (ca, sa), (cb, sb) = rows(M), rows(N)
    dt, ld = torch.bfloat16 if bf16 else torch.float32, N + pad
    D = torch.full((M, ld), 5.0, device="cuda", dtype=dt)
    (vl.vl_gemm_fp4_tn_bf16 if bf16 else vl.vl_gemm_fp4_tn)(
        H.dev(O.pack(ca)), H.dev(O.tile(sa)), H.dev(np.ldexp(np.float32(1), ea)), H.dev(O.pack(cb)), H.dev(O.tile(sb)),
        H.dev(np.ldexp(np.float32(1), eb)), D, M, N, K, ld, O.NV, alpha)
    torch.cuda.synchronize()
    A, B = (torch.from_numpy(O.values(c, s, O.NV)).cuda() for c, s in ((ca, sa), (cb, sb)))
    v = (A @ B.t()).cpu().numpy()
    step = (float(O.scale_value(np.uint8(blocks[:1]), O.NV)[0]) / 2) ** 2
    assert (A.abs() @ B.abs().t()).max() < 2 ** 24 * step         # all sums, in any order, are exact in 24 bits
    exact = np.ldexp(v * alpha, ea[:, None] + eb[None].astype(np.int64))
    with np.errstate(over="ignore"):
        want = torch.from_numpy(exact.astype(np.float32)).to(dt)
    got = D.cpu()
    assert (got[:, N:] == 5).all()
    got = got[:, :N]
    small = np.abs(exact) < 2.0 ** -126
    off = (got != want).numpy() & ~small
    assert not off.any(), (M, N, K, np.argwhere(off)[:4].tolist())
    tol = 0.75 * 2.0 ** -149 + (2.0 ** -134 if bf16 else 0)
    assert (np.abs(got.double().numpy() - exact)[small] <= tol).all(), (M, N, K)


# (M, N, K, pad): every kind of kernel, K in parts and not, D by plain stores and by TMA, ragged ends
SHAPES = [(5, 300, 512, 0), (16, 257, 4096, 1), (20, 200, 4100, 0), (60, 900, 2050, 0), (100, 700, 300, 0), (130, 600, 4096, 2),
          (200, 500, 4096, 0), (300, 9000, 2600, 0), (250, 30000, 2800, 0), (500, 8200, 700, 1)]


@pytest.mark.parametrize("M,N,K,pad", SHAPES)
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("way", ["up", "down", "all", "few"])
def test_scales_from_end_to_end(M, N, K, pad, bf16, way):
    g = np.random.default_rng(M)
    blocks = (0x68, 0x70, 0x78)  # 64, 128, 256
    if way == "up":              # large rows of A, small ones of B
        ea, eb = g.integers(60, 116, M), g.integers(-112, -60, N)
    elif way == "down":          # the other way round, over the smallest block scales
        ea, eb, blocks = g.integers(-112, -60, M), g.integers(60, 116, N), (1, 2, 4)
    elif way == "all":           # results that are infinite or nothing among them
        ea, eb = g.integers(-112, 116, M), g.integers(-112, 116, N)
    else:                        # a few such rows between ordinary ones
        ea, eb = g.integers(-8, 8, M), g.integers(-8, 8, N)
        ea[g.integers(0, M, 1 + M // 100)] = 114
        eb[g.integers(0, N, 1 + N // 200)] = -109
    product(M, N, K, ea, eb, 1.0, bf16, pad, blocks)


@pytest.mark.parametrize("M,N,K", [(20000, 300, 300), (30001, 40, 64), (6000, 1100, 500)])
@pytest.mark.parametrize("rows", [[-1], [0], [5000], [1, 127, 128, 4095, 5999]])
def test_a_few_scales_among_many_rows(M, N, K, rows):
    """Many tiles of rows, each met by some CTAs only: a row whose scale needs care anywhere among them."""
    g = np.random.default_rng(K)
    ea, eb = g.integers(-8, 8, M), g.integers(-112, -60, N)
    ea[rows] = 115
    product(M, N, K, ea, eb, 1.0, False, 0, (0x68, 0x70, 0x78))


@pytest.mark.parametrize("M,N,K,pad", [(5, 300, 512, 0), (20, 200, 4100, 0), (200, 500, 4096, 0), (300, 9000, 2600, 0)])
@pytest.mark.parametrize("alpha,ea,eb", [(2.0 ** 90, -110, 50), (-2.0 ** -100, 110, -60), (2.0 ** 127, -110, 5), (2.0 ** -149, 100, 40),
                                         (2.0 ** 70, 0, 0), (-0.375, 20, -20)])
def test_alpha_from_end_to_end(M, N, K, pad, alpha, ea, eb):
    """alpha times a row's scale out of fp32, or nearly, the result in it."""
    g = np.random.default_rng(N)
    product(M, N, K, np.full(M, ea), g.integers(0, 8, N) + eb, alpha, False, pad)
