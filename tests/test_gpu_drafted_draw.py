"""The student's half of drafted decoding: a token a sequence by verification of nothing drafted, as the example draws it."""
import numpy as np
import pytest

from oracle import draft_oracle as O
from tests import gpu_harness as H
from tests.test_gpu_drafted_step import _example, _f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,hs,V", [(1, 64, 300), (7, 256, 1001), (40, 130, 5000)])
def test_a_token_a_row(n, hs, V):
    torch, ex = H.torch_cuda(), _example()
    g = torch.Generator(device="cuda").manual_seed(n)
    w = (2 * hs ** -0.5 * torch.randn(V, hs, device="cuda", generator=g)).to(torch.bfloat16)
    step = ex.Step(ex.Head(w, torch.ones(hs, device="cuda"), torch.zeros(hs, device="cuda")), n + 2)
    heat = torch.tensor([[0.8, 0.0, 1.3][i % 3] for i in range(n)], device="cuda")
    tokens, near = torch.full((n,), -7, dtype=torch.int32, device="cuda"), 0
    for _ in range(3):
        x = torch.randn(n, hs, device="cuda", generator=g).to(torch.bfloat16)
        pick = torch.rand(n, device="cuda", generator=g)
        t = step.draw(x, heat, pick, tokens)
        torch.cuda.synchronize()
        want = O.verify(_f64(t), None, np.arange(n + 1) * 0, np.zeros(0, np.uint32), H.host(heat), np.zeros(0), H.host(pick))
        for i, (toks, _, err, margin) in enumerate(want):
            if margin < 1e-5:                        # next to a border of the running sum: either answer is right
                near += 1
                continue
            assert not err and toks == [int(H.host(tokens)[i])]
    # V - 1 borders with 1e-5 to both sides: a share of 2e-5 V of the draws at most is expected there; twice that, and 3
    assert near <= 3 + 2 * (3 * n) * 2e-5 * V
