"""Outputs that lie between the rows of their inputs: the halves of one buffer."""
import pytest

from tests import gpu_harness as H
from tests import post_plain as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,V", [(5, 77), (40, 1000), (300, 9001), (20, 20000)])
@pytest.mark.parametrize("first", [True, False])
def test_gradient_beside_the_logits(rows, V, dtype, first):
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(V)
    buf = torch.full((rows, 2 * V), 7.0, dtype=dt, device="cuda")
    x, gr = (buf[:, :V], buf[:, V:]) if first else (buf[:, V:], buf[:, :V])
    x.copy_(torch.randn(rows, V, device="cuda", generator=g) * 2)
    keep = x.clone()
    act = torch.randint(0, V, (rows,), device="cuda", generator=g)
    logp, _ = R.rows64(keep, act)
    old, adv, w = (logp - 0.1).float(), torch.randn(rows, device="cuda", generator=g), torch.ones(rows, device="cuda")
    out = {k: torch.empty(rows, device="cuda") for k in ("loss", "logp", "kl")}
    out["total"], out["grad"] = torch.empty(1, device="cuda"), gr
    f = vl.vl_policy_loss_bf16 if dtype == "bf16" else vl.vl_policy_loss
    f(x, 2 * V, rows, V, act.to(torch.int32), old, None, adv, w, 0.2, 0.28, 0.0, 1.0, gr, 2 * V, out["loss"], out["logp"],
      out["kl"], out["total"])
    torch.cuda.synchronize()
    assert torch.equal(x, keep)
    R.check_policy(out, keep, act, old, None, adv, w, 0.0, 1.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,hs", [(5, 77), (3000, 64), (2500, 1001), (900, 4096)])
def test_norm_beside_its_rows(rows, hs, dtype):
    """x, y and dx as thirds of one buffer give the bits of matrices of their own of the same stride."""
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    bf = dtype == "bf16"
    dt = torch.bfloat16 if bf else torch.float32
    fwd, bwd = (vl.vl_layernorm_fwd_bf16, vl.vl_layernorm_bwd_bf16) if bf else (vl.vl_layernorm_fwd, vl.vl_layernorm_bwd)
    src = torch.randn(rows, hs, device="cuda").to(dt)
    dy = torch.randn(rows, hs, device="cuda").to(dt)
    res = []
    for joined in (True, False):
        bufs = [torch.full((rows, 3 * hs), 7.0, dtype=dt, device="cuda") for _ in range(1 if joined else 3)] * (3 if joined else 1)
        x, y, dx = (b[:, k * hs:(k + 1) * hs] for k, b in enumerate(bufs))
        x.copy_(src)
        mu, rstd, dg, db = (torch.empty(n, device="cuda") for n in (rows, rows, hs, hs))
        fwd(x, 3 * hs, rows, hs, None, None, 1e-5, y, 3 * hs, mu, rstd)
        bwd(dy, hs, x, 3 * hs, rows, hs, None, mu, rstd, dx, 3 * hs, dg, db)
        torch.cuda.synchronize()
        assert torch.equal(x, src)
        res.append([t.clone() for t in (y, dx, mu, rstd, dg, db)])
    for a, b in zip(*res):
        assert torch.equal(a, b)
