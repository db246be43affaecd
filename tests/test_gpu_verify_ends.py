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
