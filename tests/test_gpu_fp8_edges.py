"""The quantisers' zeros, and few-row products of more tiles than CTAs.  Tolerances as in test_gpu_fp8.py."""
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


@pytest.mark.parametrize("M", [3, 20, 50])
def test_product_of_few_rows_and_many_tiles(M):
    """More 128-row tiles of the plane than two CTAs an SM take at once, and more than one batch of scales."""
    product(M, 40001, 1040)
