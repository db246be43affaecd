"""Random numbers of exactly 1 (a draw in [0, 1) rounded up on its way to fp32)."""
import numpy as np
import pytest

from tests import gpu_harness as H

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("draft", [True, False])
def test_a_token_that_is_certain_and_refused_is_drawn(draft):
    """u = 1 refuses a token whose probability is 1; nothing is left of the weights then, so p itself is drawn from."""
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    V = 2500
    t = np.full((6, V), -np.inf, np.float32)
    at = np.array([5, 9, 1030, 7, 2499, 11])
    t[np.arange(6), at] = 2.0
    tokens, acc = torch.full((6,), 77, dtype=torch.int32, device="cuda"), torch.full((3,), 77, dtype=torch.int32, device="cuda")
    lp, err = torch.full((6,), 77.0, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    x = H.dev(t)
    vl.vl_verify_draft(x, V, x[::2].contiguous() if draft else None, V, V, H.dev(np.arange(4, dtype=np.int64)), 3, 3,
                       H.dev(at[::2].astype(np.uint32)), None, H.dev(np.ones(3, np.float32)), H.dev(np.float32([0, 0.5, 1])), tokens, acc,
                       lp, err)
    torch.cuda.synchronize()
    none = 0xFFFFFFFF
    assert H.host(tokens).view(np.uint32).tolist() == [5, none, 1030, none, 2499, none]
    assert H.host(acc).tolist() == [0, 0, 0] and (H.host(lp) == 0).all() and int(H.host(err)[0]) == 0


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_u_of_0_accepts_whatever_has_a_probability(draft, dtype):
    """0 < p, however small p is: e^-100 and e^-700 (not in fp32, nor their ratios to q), but not 0."""
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    V, low = 2500, np.float32([-100, -700, -800, -np.inf])
    t = np.zeros((8, V), np.float32)
    t[:, 1] = 50                                                 # about all of p
    t[::2, 3] = 50 + low
    y = np.zeros((4, V), np.float32)
    y[:, 3] = 60                                                 # about all of q
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    tokens, acc = torch.full((8,), 77, dtype=torch.int32, device="cuda"), torch.full((4,), 77, dtype=torch.int32, device="cuda")
    (vl.vl_verify_draft_bf16 if dtype == "bf16" else vl.vl_verify_draft)(
        H.dev(t).to(dt), V, H.dev(y).to(dt) if draft else None, V, V, H.dev(np.arange(5, dtype=np.int64)), 4, 4,
        H.dev(np.full(4, 3, np.uint32)), None, H.dev(np.zeros(4, np.float32)), H.dev(np.full(4, 0.5, np.float32)), tokens, acc)
    torch.cuda.synchronize()
    assert H.host(acc).tolist() == [1, 1, 0, 0]
    none = 0xFFFFFFFF
    assert H.host(tokens).view(np.uint32).tolist() == [3, 1, 3, 1, 1, none, 1, none]
