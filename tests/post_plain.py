"""Float64 evaluation of the policy and preference losses over many rows, in elementary torch
operations on the GPU, a block of rows at a time, with the tolerances of test_gpu_post_loss.py:
a log-probability within delta = 4 ulp(max(|s[a] - m|, ln S, 1)) + 64 * 2^-24 plus 2^-21 of what
enters it, whatever follows by its derivative plus 2^-21 of its terms, gradients 1e-6 of the row's
factor besides; a bf16 gradient between the bf16 roundings of the ends of the fp32 interval.
"""
import torch

EPS = 2.0 ** -24
U = 2.0 ** -21
BLOCK = 1024


def _ulp(v):
    v = v.float().abs()
    return (torch.nextafter(v, torch.full_like(v, float("inf"))) - v).double()


def _near(got, want, tol, what):
    got, want = got.double(), want.double()
    ok = (got == want) | (got.isnan() & want.isnan()) | ((got - want).abs() <= tol)
    assert bool(ok.all()), (what, int((~ok).sum()), (~ok).nonzero()[:4].tolist(), got[~ok][:4].tolist(), want[~ok][:4].tolist())


def _near_rounded(got, want, tol, what):
    if got.dtype != torch.bfloat16:
        return _near(got, want, tol, what)
    lo, hi = ((want + s * tol).float().to(torch.bfloat16).double() for s in (-1, 1))
    got = got.double()
    ok = ((got >= lo) & (got <= hi)) | (got.isnan() & want.isnan())
    assert bool(ok.all()), (what, int((~ok).sum()), (~ok).nonzero()[:4].tolist(), got[~ok][:4].tolist(), want[~ok][:4].tolist())


def rows64(x, pick):
    """(logp of column pick, its tolerance delta) of every row; rows whose pick is out of range get 0."""
    n, V = x.shape
    logp, delta = (torch.zeros(n, dtype=torch.float64, device=x.device) for _ in range(2))
    for a in range(0, n, BLOCK):
        b = x[a:a + BLOCK].double()
        ok = pick[a:a + BLOCK] < V
        xa = b.gather(1, torch.where(ok, pick[a:a + BLOCK], 0)[:, None])[:, 0]
        m = b.amax(1)
        lnS = (b - m[:, None]).exp().sum(1).log()
        logp[a:a + BLOCK] = torch.where(ok, (xa - m) - lnS, 0.0)
        delta[a:a + BLOCK] = 4 * _ulp(torch.maximum((xa - m).abs(), lnS).clamp(min=1.0)) + 64 * EPS
    return logp, delta


def check_gradient(grad, x, pick, factor, tol, what="gradient"):
    """grad against factor ([j == pick] - softmax(x)) of each row; factor 0 is a row of zeros."""
    n, V = x.shape
    for a in range(0, n, BLOCK):
        live = factor[a:a + BLOCK] != 0
        b = torch.where(live[:, None], x[a:a + BLOCK].double(), 0.0)
        want = torch.softmax(b, 1).neg_()
        at = torch.where(live, pick[a:a + BLOCK], 0)
        want.scatter_add_(1, at[:, None], torch.ones_like(want[:, :1]))
        want *= factor[a:a + BLOCK, None]
        _near_rounded(grad[a:a + BLOCK], want, tol[a:a + BLOCK, None], what)


def check_policy(got, x, act, old, ref, adv, w, kl_coef, scale, lo=0.2, hi=0.28):
    """got: loss, logp, kl [n], total [1], grad [n][V], all on the GPU; x as the call got it (before a
    gradient in place), with finite rows wherever w != 0."""
    lo, hi, kl_coef, scale = (float(torch.tensor(v, dtype=torch.float32)) for v in (lo, hi, kl_coef, scale))
    live = (w != 0) & (act < x.shape[1])
    bad = (w != 0) & (act >= x.shape[1])
    old, adv, w64 = old.double(), adv.double(), w.double()
    logp, d = rows64(torch.where(live[:, None], x, torch.zeros_like(x)), act)
    d = d + U * (1 + logp.abs() + old.abs())
    r = (logp - old).exp()
    f, h = r * adv, r.clamp(1 - lo, 1 + hi) * adv
    each, dl = -torch.minimum(f, h), torch.where(f <= h, -f, 0.0)
    q = torch.zeros_like(logp) if ref is None else ref.double() - logp
    kl = torch.expm1(q) - q
    each, dl = each + kl_coef * kl, dl - kl_coef * torch.expm1(q)
    nan = torch.full_like(logp, float("nan"))
    loss, G = torch.where(live, w64 * each, 0.0), torch.where(live, w64 * dl, 0.0)
    eq, ra = q.exp(), r * adv.abs()
    _near(got["logp"], torch.where(bad, nan, torch.where(live, logp, 0.0)), d, "logp")
    _near(got["kl"], torch.where(live, kl, 0.0), torch.where(live, (eq - 1).abs() * d + (eq + q.abs()) * U, 0.0), "kl")
    tol = torch.where(live, w64.abs() * (ra * (d + U) + abs(kl_coef) * ((eq - 1).abs() * d + (eq + q.abs()) * U)), 0.0)
    _near(got["loss"], torch.where(bad, nan, loss), tol, "loss")
    if not bool(bad.any()):
        assert abs(float(got["total"]) - float(loss.sum())) <= float(tol.sum()) + 2 * EPS * abs(float(loss.sum()))
    else:
        assert bool(got["total"].isnan())
    # the part of the factor that the clip takes away does not count
    dG = scale * w64.abs() * (ra + abs(kl_coef) * (ref is not None) * eq) * (d + U)
    check_gradient(got["grad"], x, act, scale * G, torch.where(live, dG + 1e-6 * (scale * G).abs(), 0.0))


def check_preference(got, x, lab, w, start, npairs, ref, beta, smooth, kind, scale):
    """got: loss, margin [npairs], seq [2 npairs], mean [1], grad [n][V]; kind 0 (sigmoid) or 1 (squared);
    start a list, its sequences next to one another."""
    n, V = x.shape
    beta, smooth, scale = (float(torch.tensor(v, dtype=torch.float32)) for v in (beta, smooth, scale))
    live = w != 0
    lost = live & (lab >= V)
    w64 = torch.where(live, w.double(), 0.0)
    logp, d = rows64(torch.where((live & ~lost)[:, None], x, torch.zeros_like(x)), lab)
    dlp = w64.abs() * (d + U * logp.abs())
    seq, tol, bad = (torch.stack([v[a:b].sum() for a, b in zip(start, start[1:])]) for v in (w64 * logp, dlp, lost.double()))
    bad = (bad[:npairs] + bad[npairs:]) > 0
    one = torch.tensor([bool(lost[a:b].any()) for a, b in zip(start, start[1:])], device=x.device)
    nan = torch.full_like(seq, float("nan"))
    _near(got["seq"], torch.where(one, nan, seq), tol + 2 * EPS * seq.abs(), "seq")
    lift = seq - (0 if ref is None else ref.double())
    gap, tol = lift[:npairs] - lift[npairs:], tol[:npairs] + tol[npairs:]
    _near(got["margin"], torch.where(bad, nan[:npairs], beta * gap), beta * tol + 4 * EPS * (beta * gap).abs(), "margin")
    tol = tol + 4 * EPS * gap.abs()
    if kind == 0:
        ls = torch.nn.functional.logsigmoid
        loss = -(1 - smooth) * ls(beta * gap) - smooth * ls(-beta * gap)
        slope, bend = beta * (smooth * torch.sigmoid(beta * gap) - (1 - smooth) * torch.sigmoid(-beta * gap)), beta * beta / 4
    else:
        z = gap - 1 / (2 * beta)
        loss, slope, bend = z * z, 2 * z, 2.0
    dl = slope.abs() * tol + bend * tol ** 2 + U * (loss.abs() + (kind == 0))
    _near(got["loss"], torch.where(bad, nan[:npairs], loss), dl, "loss")
    if not bool(bad.any()):
        assert abs(float(got["mean"]) - float(loss.mean())) <= float(dl.mean()) + 1e-6 * abs(float(loss.mean()))
    else:
        assert bool(got["mean"].isnan())
    factor, ftol = torch.zeros_like(w64), torch.zeros_like(w64)
    for s in range(2 * npairs):
        i, sl = s % npairs, slice(start[s], start[s + 1])
        if not bool(bad[i]):
            factor[sl] = (1 if s < npairs else -1) * scale * slope[i] * w64[sl]
            c = scale * w64[sl].abs()
            ftol[sl] = c * (bend * tol[i] + 2 * U * slope[i].abs() + U * beta * (kind == 0)) + 1e-6 * c * slope[i].abs()
    check_gradient(got["grad"], x, lab, factor, ftol)
