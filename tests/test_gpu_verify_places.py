"""Sequences of odd vocabularies in batches that put their rows at other places within 16 bytes."""
import numpy as np
import pytest

from tests import gpu_harness as H
from tests.test_gpu_verify import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [2999, 3001, 3002])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("draft", [True, False])
def test_parts_of_a_batch(V, dtype, draft):
    """The same bits where the rows stand at the same place within 16 bytes; elsewhere the same tokens (random numbers are off the
    borders), and log-probabilities each of which is off by at most 4 ulp + 2^-18 (of sizes below 32: an ulp is 2^-19)."""
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    n, k = 90, 3
    t, y, s, tok, h, u, p = make([k] * n, V, 31, temp=[0.8, 1.3], near=0.4, draft=draft, dtype=dtype)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    t, y = H.dev(t).to(dt), H.dev(y).to(dt) if draft else None
    tok, h, u, p = H.dev(tok).view(torch.int32), H.dev(h), H.dev(u), H.dev(p)
    per = 16 // t.element_size()                                   # sequences after which the places come again

    def call(a, b):
        # a buffer of its own, so that the part's first row begins at 16 bytes
        m = b - a
        x, q = t[a * (k + 1):b * (k + 1)].clone(), y[a * k:b * k].clone() if draft else None
        out = [torch.empty(m * (k + 1), dtype=torch.int32, device="cuda"), torch.empty(m, dtype=torch.int32, device="cuda"),
               torch.empty(m * (k + 1), device="cuda")]
        (vl.vl_verify_draft_bf16 if dtype == "bf16" else vl.vl_verify_draft)(
            x, V, q, V, V, H.dev(np.arange(m + 1, dtype=np.int64) * k), m, m * k, tok[a * k:b * k], h[a:b], u[a * k:b * k], p[a:b], *out)
        torch.cuda.synchronize()
        return out

    whole = call(0, n)
    for a, b in ((0, 1), (per, per + 3), (1, 2), (5, 30), (2 * per, n), (3, 80)):
        part = call(a, b)
        assert torch.equal(part[0], whole[0][a * (k + 1):b * (k + 1)]) and torch.equal(part[1], whole[1][a:b])
        off = (part[2] - whole[2][a * (k + 1):b * (k + 1)]).abs().max()
        assert off == 0 if a % per == 0 else off <= 2 * (4 * 2.0 ** -19 + 2.0 ** -18)
