"""Policy and preference losses over long rows, compared with float64 (post_plain.py)."""
import pytest

from tests import gpu_harness as H
from tests import post_plain as R

pytestmark = pytest.mark.gpu


def _tensors(n, V, dtype, seed, ld=None):
    """Logits in rows of stride ld (NaN between), with a confident pick in three rows of ten."""
    torch = H.torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(seed)
    ld = ld or V
    buf = torch.full((n, ld), float("nan"), dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device="cuda")
    x = buf[:, :V]
    pick = torch.randint(0, V, (n,), device="cuda", generator=g)
    for a in range(0, n, R.BLOCK):
        b = torch.randn(min(R.BLOCK, n - a), V, device="cuda", generator=g) * 3
        sure = (torch.rand(b.shape[0], device="cuda", generator=g) < 0.3).float() * 8
        b.scatter_add_(1, pick[a:a + R.BLOCK, None], sure[:, None])
        x[a:a + R.BLOCK] = b.to(x.dtype)
    return g, buf, x, pick


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [20000, 70000])
def test_few_long_rows_some_of_which_do_not_count(V, dtype):
    """Fewer rows than CTAs, half of them of weight 0, in both losses."""
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    n, bf = 30, dtype == "bf16"
    g, buf, x, act = _tensors(n, V, dtype, V)
    at = torch.arange(n, device="cuda")
    w = (at % 2).float()
    x[w == 0] = float("nan")
    keep = x.clone()
    logp, _ = R.rows64(torch.where((w != 0)[:, None], x, torch.zeros_like(x)), act)
    old, adv = (logp + 0.1).float(), torch.randn(n, device="cuda", generator=g)
    out = {k: torch.full((n,), 9.0, device="cuda") for k in ("loss", "logp", "kl")}
    out["total"], out["grad"] = torch.empty(1, device="cuda"), torch.empty_like(x)
    f = vl.vl_policy_loss_bf16 if bf else vl.vl_policy_loss
    f(x, V, n, V, act.to(torch.int32), old, None, adv, w, 0.2, 0.28, 0.0, 1.0, out["grad"], V, out["loss"], out["logp"], out["kl"],
      out["total"])
    torch.cuda.synchronize()
    R.check_policy(out, keep, act, old, None, adv, w, 0.0, 1.0)
    start = [0, 9, 15, 22, n]
    out = {k: torch.full((m,), 9.0, device="cuda") for k, m in (("loss", 2), ("margin", 2), ("seq", 4), ("mean", 1))}
    f = vl.vl_preference_loss_bf16 if bf else vl.vl_preference_loss
    f(x, V, n, V, act.to(torch.int32), w, torch.tensor(start, device="cuda"), 2, None, 0.05, 0.0, 0, 0.5, x, V, out["loss"],
      out["margin"], out["seq"], out["mean"])
    torch.cuda.synchronize()
    out["grad"] = x
    R.check_preference(out, keep, act, w, start, 2, None, 0.05, 0.0, 0, 0.5)
