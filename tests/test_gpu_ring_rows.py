"""Policy and preference losses over as many long rows as turn every buffer of the ring kernel over:
more than 32 rows a CTA or cluster (a second batch of token data), more than 8 (the buffers of the warps'
partials), more than 96 (a second window of rows), with rows of weight 0 between, bad labels, rows
of different alignment, in place and apart.  Compared with float64 (post_plain.py)."""
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


# one CTA a row and a second window; clusters of two CTAs and a second window; clusters of two and three CTAs and a
# second batch; rows of every alignment
POLICY = [("bf16", 15000, 8200, 8200), ("f32", 6000, 8201, 8201), ("bf16", 7500, 62000, 62000), ("f32", 2700, 46100, 46104),
          ("f32", 2000, 100000, 100000), ("bf16", 1200, 9001, 9003)]


@pytest.mark.parametrize("dtype,n,V,ld", POLICY)
def test_policy_of_many_long_rows(dtype, n, V, ld):
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    g, buf, x, act = _tensors(n, V, dtype, n + V, ld)
    logp, _ = R.rows64(x, act)
    d = 0.25 * torch.randn(n, device="cuda", generator=g)
    for e in (-0.22314355, 0.24686008):                      # the clip's edges, where the gradient jumps
        d = torch.where((d - e).abs() < 4e-3, d + 0.01, d)
    old, ref = (logp - d).float(), (logp + 0.4 * torch.randn(n, device="cuda", generator=g)).float()
    adv = torch.randn(n, device="cuda", generator=g)
    at = torch.arange(n, device="cuda")
    # prompts (runs of rows that do not count), single ones between, and bad actions
    w = ((at % 211 >= 40) & (at % 7 != 3)).float() * (0.5 + torch.rand(n, device="cuda", generator=g)) / n
    act[at % 997 == 500] = V
    act[at % 997 == 501] = 0xFFFFFFFF
    bad = int(((w != 0) & (act >= V)).sum())
    x[(w == 0) & (at % 5 == 0)] = float("nan")               # rows that do not count may hold anything
    keep = x.clone()
    act32 = torch.where(act >= 1 << 31, act - (1 << 32), act).to(torch.int32)
    grad = torch.full_like(buf, 3.0)
    f = vl.vl_policy_loss_bf16 if dtype == "bf16" else vl.vl_policy_loss
    runs = []
    for gr in (grad, buf):                                   # apart, then in place
        out = {k: torch.full((n,), 9.0, device="cuda") for k in ("loss", "logp", "kl")}
        out["total"], err = torch.full((1,), 9.0, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        f(buf, ld, n, V, act32, old, ref, adv, w, 0.2, 0.28, 0.04, 1.0, gr, ld, out["loss"], out["logp"], out["kl"],
          out["total"], err)
        torch.cuda.synchronize()
        assert int(err) == bad
        out["grad"] = gr[:, :V]
        runs.append(out)
    assert bool((grad[:, V:] == 3).all())
    R.check_policy(runs[0], keep, act, old, ref, adv, w, 0.04, 1.0)
    for k in runs[0]:
        a, b = runs[0][k], runs[1][k]
        assert bool(((a == b) | (a.isnan() & b.isnan())).all()), k


# one CTA a row and several windows; clusters in the first pass (160 rows of 128256 columns)
PREF = [("bf16", 1200, 8200, 8200, 12, 1), ("f32", 1300, 8201, 8203, 9, 0), ("bf16", 15600, 8200, 8200, 60, 0),
        ("f32", 160, 128256, 128256, 4, 0), ("f32", 6000, 9000, 9000, 30, 1), ("bf16", 330, 128256, 128256, 8, 0)]


@pytest.mark.parametrize("dtype,n,V,ld,npairs,kind", PREF)
def test_preference_of_many_long_rows(dtype, n, V, ld, npairs, kind):
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    g, buf, x, lab = _tensors(n, V, dtype, n + V, ld)
    # sequences of unequal lengths, one of them empty, rows after the last one
    cut = sorted(torch.randperm(n - 20, generator=torch.Generator().manual_seed(n))[:2 * npairs].tolist())
    start = [0] + cut
    start[2] = start[1]
    at = torch.arange(n, device="cuda")
    first = torch.tensor(start, device="cuda")
    seq = torch.searchsorted(first, at, right=True) - 1
    within = at - first[seq]
    w = ((within >= 5) & (at % 11 != 4)).float() * (0.5 + torch.rand(n, device="cuda", generator=g))
    w[start[-1]:] = 1.0                                      # of no sequence
    if kind == 1:
        w = w / 40
    long = max(range(2 * npairs), key=lambda s: start[s + 1] - start[s])
    lab[start[long] + 6], w[start[long] + 6] = V, 1.0        # its pair is lost
    lab[n - 1] = V + 5                                       # counted, of no sequence
    x[(w == 0) & (at % 5 == 0)] = float("nan")
    keep = x.clone()
    live = torch.where(lab < V, lab, 0)
    logp, _ = R.rows64(torch.where((w != 0)[:, None], x, torch.zeros_like(x)), live)
    pi = torch.stack([(w.double() * logp)[a:b].sum() for a, b in zip(start, start[1:])])
    ref = (pi + 2 * torch.randn(2 * npairs, device="cuda", generator=g)).float()
    lab32, start_d = lab.to(torch.int32), first
    beta, smooth = 0.1, 0.1 if kind == 0 else 0.0
    grad = torch.full_like(buf, 3.0)
    f = vl.vl_preference_loss_bf16 if dtype == "bf16" else vl.vl_preference_loss
    runs = []
    for gr in (grad, buf):
        out = {k: torch.full((m,), 9.0, device="cuda") for k, m in (("loss", npairs), ("margin", npairs), ("seq", 2 * npairs), ("mean", 1))}
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        ws = torch.full((vl.vl_preference_workspace_bytes(n, npairs),), 0xFF, dtype=torch.uint8, device="cuda")
        f(buf, ld, n, V, lab32, w, start_d, npairs, ref, beta, smooth, kind, 1.0 / npairs, gr, ld, out["loss"], out["margin"],
          out["seq"], out["mean"], err, workspace=ws)
        torch.cuda.synchronize()
        assert int(err) == 2
        out["grad"] = gr[:, :V]
        runs.append(out)
    assert bool((grad[:, V:] == 3).all())
    R.check_preference(runs[0], keep, lab, w, start, npairs, ref, beta, smooth, kind, 1.0 / npairs)
    assert int(runs[0]["loss"].isnan().sum()) == 1 and not bool(runs[0]["grad"][start[-1]:].any())
    for k in runs[0]:
        a, b = runs[0][k], runs[1][k]
        assert bool(((a == b) | (a.isnan() & b.isnan())).all()), k


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
