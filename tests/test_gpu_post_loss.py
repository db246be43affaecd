"""Policy and preference losses on the GPU against the float64 definitions.

Tolerances, from the arithmetic.  A row's log-probability is (s[a] - m) - ln S in fp32: within
delta = 4 ulp(max(|s[a] - m|, ln S, 1)) + 64 * 2^-24.  A ratio or exponential of it is off by
delta relatively, plus 2^-21 for the function and the products around it; a softmax value of
the gradient by 1e-6 absolutely (the bar of the other losses' gradients).  Sequence sums add
their rows' errors.  A bf16 gradient is that value rounded once: it lies between the bf16
roundings of the ends of the fp32 interval.
"""
import numpy as np
import pytest

from oracle import post_oracle as O
from tests import gpu_harness as H

pytestmark = pytest.mark.gpu

U = 2.0 ** -21


def _place(a, ld, off, dtype, fill=float("nan")):
    """Rows of a in a device buffer with stride ld, `off` elements in; everything else is `fill`."""
    torch = H.torch_cuda()
    n, V = a.shape
    buf = torch.full((off + max(n, 1) * ld + 16,), fill, dtype=dtype, device="cuda")
    view = buf[off:off + n * ld].view(n, ld) if n else buf[:0].view(0, ld)
    view[:, :V] = torch.from_numpy(np.ascontiguousarray(a)).cuda().to(dtype)
    return buf, view


def _wide(view, V):
    return view[:, :V].float().cpu().numpy().astype(np.float64)


def _delta(x, act, w):
    d = np.zeros(len(act))
    for t in range(len(act)):
        if w[t] != 0 and act[t] < x.shape[1]:
            m = x[t].max()
            lnS = np.log(np.exp(x[t] - m).sum())
            d[t] = 4 * H.ulp(max(abs(x[t, act[t]] - m) if np.isfinite(x[t, act[t]]) else 1.0, lnS, 1.0)) + 64 * H.EPS
    return d


def _check(got, want, tol, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        bad = ~(same | (np.abs(got - want) <= tol))
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4])


def check_rounded(got, want, tol, dtype, what):
    """fp32 values within tol of want; bf16 ones between the roundings of want - tol and want + tol."""
    if dtype != "bf16":
        return _check(got, want, tol, what)
    torch = H.torch_cuda()
    lo, hi = (torch.from_numpy(want + s * np.broadcast_to(tol, want.shape)).float().to(torch.bfloat16).double().numpy()
              for s in (-1.0, 1.0))
    bad = ~(((got >= lo) & (got <= hi)) | (got == want) | (np.isnan(got) & np.isnan(want)))
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4])


def _inputs(n, V, seed, dtype):
    torch = H.torch_cuda()
    g = np.random.default_rng(seed)
    x = (g.normal(size=(n, V)) * 3).astype(np.float32)
    act = g.integers(0, V, n).astype(np.uint32)
    sure = g.random(n) < 0.3
    x[np.nonzero(sure)[0], act[sure]] += 8
    x = torch.from_numpy(x).to(dtype).float().numpy()
    x64 = x.astype(np.float64)
    lp = np.array([O.row_logp(x64[t], act[t])[0] for t in range(n)])
    old = lp - g.normal(size=n) * 0.25
    for e in (np.log(0.8), np.log(1.28)):                  # away from the jumps of the gradient
        near = np.abs((lp - old) - e) < 4e-3
        old[near] -= 0.01
    return g, x, act, old.astype(np.float32), (lp + g.normal(size=n) * 0.5).astype(np.float32)


def run_policy(x, act, old, ref, adv, w, kl, scale, dtype, ld=None, ldg=None, off=0, goff=0, inplace=False, want_grad=True,
               lo=0.2, hi=0.28, stream=None):
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    n, V = x.shape
    ld, ldg = ld or V, ldg or V
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    _, xv = _place(x, ld, off, dt)
    if inplace:
        gv, ldg, gbuf = xv, ld, None
    elif want_grad:
        gbuf, gv = _place(np.full((n, V), 7.0, np.float32), ldg, goff, dt, fill=3.0)
    else:
        gv = None
    dev = [H.dev(a) if a is not None else None for a in (act, old, ref, adv, w)]
    loss, logp, klv = (torch.full((max(n, 1),), 9.0, device="cuda") for _ in range(3))
    total, err = torch.full((1,), 9.0, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    f = vl.vl_policy_loss_bf16 if dtype == "bf16" else vl.vl_policy_loss
    f(xv.data_ptr(), ld, n, V, dev[0], dev[1], dev[2], dev[3], dev[4], lo, hi, kl, scale,
      None if gv is None else gv.data_ptr(), ldg, loss, logp, klv, total, err, stream)
    torch.cuda.synchronize()
    if gv is not None and not inplace:                     # nothing outside the rows is written
        assert bool((gbuf[:goff] == 3).all()) and bool((gv[:, V:] == 3).all()) and bool((gbuf[goff + n * ldg:] == 3).all())
    return dict(loss=H.host(loss)[:n], logp=H.host(logp)[:n], kl=H.host(klv)[:n], total=float(total[0]), err=int(err[0]),
                grad=None if gv is None else _wide(gv, V))


def check_policy(got, x, act, old, ref, adv, w, kl, scale, dtype, lo=0.2, hi=0.28):
    x = x.astype(np.float64)
    lo, hi, kl, scale = (float(np.float32(v)) for v in (lo, hi, kl, scale))
    want = O.policy(x, act, old, ref, adv, w, lo, hi, kl, scale)
    d = _delta(x, act, w)
    with np.errstate(invalid="ignore", over="ignore"):
        r = np.exp(want["logp"] - old) * np.abs(adv)
        q = np.zeros(len(w)) if ref is None else ref - want["logp"]
        eq = np.exp(q)
    d = d + U * (1 + np.abs(np.nan_to_num(want["logp"])) + np.abs(old))     # the differences' own rounding
    _check(got["logp"], want["logp"], d, "logp")
    _check(got["kl"], want["kl"], np.where(w != 0, np.abs(eq - 1) * d + (eq + np.abs(q)) * U, 0), "kl")
    dl = np.abs(w) * (r * (d + U) + abs(kl) * (np.abs(eq - 1) * d + (eq + np.abs(q)) * U))
    _check(got["loss"], want["loss"], np.nan_to_num(dl), "loss")
    if not np.isnan(want["total"]):
        assert abs(got["total"] - want["total"]) <= np.nan_to_num(dl).sum() + 2 * H.EPS * abs(want["total"])
    else:
        assert np.isnan(got["total"])
    if got["grad"] is not None:
        dG = scale * np.abs(w) * (r + abs(kl) * (ref is not None) * eq) * (d + U)
        tol = (np.nan_to_num(dG) + 1e-6 * np.abs(scale * np.nan_to_num(want["G"])))[:, None]
        check_rounded(got["grad"], want["grad"], tol, dtype, "gradient")


SHAPES = [(1, 1), (3, 2), (5, 7), (2, 31), (64, 1024), (9, 4099), (7, 8192), (5, 32003), (3, 50257), (2, 128256), (2, 200001),
          (2, 245760)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,V", SHAPES)
def test_policy(n, V, dtype):
    torch = H.torch_cuda()
    g, x, act, old, ref = _inputs(n, V, n + V, torch.bfloat16 if dtype == "bf16" else torch.float32)
    adv = g.normal(size=n).astype(np.float32)
    w = (g.random(n) + 0.1).astype(np.float32) / n
    if n > 2:
        w[1] = 0
    got = run_policy(x, act, old, ref, adv, w, 0.04, 1.5, dtype)
    assert got["err"] == 0
    check_policy(got, x, act, old, ref, adv, w, 0.04, 1.5, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_policy_rows_past_the_one_pass_limit(dtype):
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    V = vl.VL_POLICY_ONEPASS_COLS + 5003
    g, x, act, old, ref = _inputs(2, V, 77, torch.bfloat16 if dtype == "bf16" else torch.float32)
    adv, w = np.array([1.0, -1.0], np.float32), np.array([0.5, 0.5], np.float32)
    check_policy(run_policy(x, act, old, ref, adv, w, 0.04, 1.0, dtype), x, act, old, ref, adv, w, 0.04, 1.0, dtype)
    got = run_policy(x, act, old, ref, adv, w, 0.04, 1.0, dtype, inplace=True, ld=V + 3)
    check_policy(got, x, act, old, ref, adv, w, 0.04, 1.0, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,ld,off,ldg,goff", [(1000, 1003, 1, 1003, 1), (1000, 1001, 3, 1005, 2), (4097, 4097, 0, 4104, 0),
                                               (33001, 33001, 5, 33001, 5), (33001, 33004, 1, 33008, 3), (5, 9, 2, 6, 1)])
def test_policy_strides_and_alignment(V, ld, off, ldg, goff, dtype):
    torch = H.torch_cuda()
    n = 6
    g, x, act, old, ref = _inputs(n, V, V, torch.bfloat16 if dtype == "bf16" else torch.float32)
    act[:3] = [0, V - 1, V // 2]
    old = (np.array([O.row_logp(x[t].astype(np.float64), act[t])[0] for t in range(n)]) + 0.1).astype(np.float32)
    adv, w = g.normal(size=n).astype(np.float32), np.full(n, 0.25, np.float32)
    a = (x, act, old, None, adv, w, 0.0, 1.0, dtype)
    check_policy(run_policy(*a, ld=ld, off=off, ldg=ldg, goff=goff), *a)
    check_policy(run_policy(*a, ld=ld, off=off, inplace=True), *a)
    got = run_policy(*a, ld=ld, off=off, want_grad=False)
    assert got["grad"] is None
    check_policy(got, *a)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [37, 3000, 40000])
def test_policy_masks_infinities_and_bad_actions(V, dtype):
    torch = H.torch_cuda()
    n = 12
    g, x, act, old, ref = _inputs(n, V, 3 * V, torch.bfloat16 if dtype == "bf16" else torch.float32)
    adv, w = g.normal(size=n).astype(np.float32), np.full(n, 1 / 8, np.float32)
    w[[0, 4, 11]] = 0
    x[0], x[4, 3] = np.nan, np.inf                          # rows that do not count may hold anything
    act[11] = 0xFFFFFFFF
    x[2, :V // 2] = -np.inf                                 # a masked vocabulary
    x[3] = np.finfo(np.float32).min if dtype == "f32" else -3e38   # every logit at the type's lowest value
    x = torch.from_numpy(x).to(torch.bfloat16 if dtype == "bf16" else torch.float32).float().numpy()
    x[5] = -np.inf                                          # one value left
    x[5, act[5]] = 2.0
    act[2], act[7], act[8] = V - 1, V, 0xFFFFFFFE           # the last two are bad
    for t in (2, 3, 5):
        old[t] = O.row_logp(x[t].astype(np.float64), act[t])[0] + 0.05
        ref[t] = old[t] - 0.2
    adv[6], old[6], ref[6] = 1.0, old[6] - 60.0, old[6] - 80.0     # a vast ratio that the clip takes away
    adv[9] = 0.0
    got = run_policy(x, act, old, ref, adv, w, 0.04, 1.0, dtype)
    assert got["err"] == 2 and np.isnan(got["loss"][[7, 8]]).all() and not got["grad"][[0, 4, 7, 8, 11]].any()
    check_policy(got, x, act, old, ref, adv, w, 0.04, 1.0, dtype)
    w[[7, 8]] = 0
    got = run_policy(x, act, old, ref, adv, w, 0.0, 1.0, dtype, inplace=True)
    assert got["err"] == 0 and got["kl"][1] > 0            # reported though it is not in the loss
    check_policy(got, x, act, old, ref, adv, w, 0.0, 1.0, dtype)
    none = run_policy(x, act, old, ref, adv, np.zeros(n, np.float32), 0.04, 1.0, dtype)
    assert none["total"] == 0 and not none["grad"].any() and not none["loss"].any() and not none["logp"].any()


def test_policy_nan_row_stays_in_its_row():
    n, V = 5, 20000
    g, x, act, old, ref = _inputs(n, V, 8, H.torch_cuda().float32)
    adv, w = np.ones(n, np.float32), np.ones(n, np.float32)
    x[2, 17] = np.nan
    got = run_policy(x, act, old, ref, adv, w, 0.1, 1.0, "f32")
    assert np.isnan(got["loss"][2]) and np.isnan(got["grad"][2]).all() and np.isnan(got["total"])
    keep = [0, 1, 3, 4]
    part = {k: (v[keep] if isinstance(v, np.ndarray) else v) for k, v in got.items()}
    part["total"] = float(got["loss"][keep].astype(np.float64).sum())
    check_policy(part, x[keep], act[keep], old[keep], ref[keep], adv[keep], w[keep], 0.1, 1.0, "f32")


def test_policy_many_rows_other_stream_and_repeats():
    """More rows than CTAs, in place and apart, on a stream of its own: the same bits every time."""
    torch = H.torch_cuda()
    for n, V, dtype in ((700, 3001, "f32"), (701, 20000, "bf16"), (400, 66000, "bf16")):
        g, x, act, old, ref = _inputs(n, V, n, torch.bfloat16 if dtype == "bf16" else torch.float32)
        adv, w = g.normal(size=n).astype(np.float32), (g.random(n) < 0.7).astype(np.float32) / n
        s = torch.cuda.Stream()
        a = run_policy(x, act, old, ref, adv, w, 0.02, 1.0, dtype, stream=s)
        b = run_policy(x, act, old, ref, adv, w, 0.02, 1.0, dtype, inplace=True)
        check_policy(a, x, act, old, ref, adv, w, 0.02, 1.0, dtype)
        assert np.array_equal(a["grad"], b["grad"]) and np.array_equal(a["loss"], b["loss"]) and a["total"] == b["total"]


def test_policy_offsets_past_32_bits():
    """The rows of a buffer of more than 2^32 elements: the last one is right."""
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    n, V, ld = 3, 1000, (1 << 31) + 8
    buf = torch.zeros(2 * ld + V, dtype=torch.bfloat16, device="cuda")
    g, x, act, old, ref = _inputs(n, V, 4, torch.bfloat16)
    for t in range(n):
        buf[t * ld:t * ld + V] = torch.from_numpy(x[t]).cuda().to(torch.bfloat16)
    adv, w = np.ones(n, np.float32), np.ones(n, np.float32)
    loss = torch.empty(n, device="cuda")
    args = [H.dev(a) for a in (act, old, ref, adv, w)]
    vl.vl_policy_loss_bf16(buf, ld, n, V, *args, 0.2, 0.28, 0.1, 1.0, buf, ld, loss)
    torch.cuda.synchronize()
    got = dict(loss=H.host(loss), grad=np.stack([buf[t * ld:t * ld + V].float().cpu().numpy() for t in range(n)]))
    assert not bool(buf[V:V + 4096].any())
    want = O.policy(x.astype(np.float64), act, old, ref, adv, w, *(float(np.float32(v)) for v in (0.2, 0.28, 0.1, 1.0)))
    assert np.abs(got["loss"] - want["loss"]).max() < 1e-4
    assert np.abs(got["grad"] - want["grad"]).max() < 1e-2


# ---------------------------------------------------------------- preference


def run_pref(x, lab, w, start, npairs, ref, beta, smooth, kind, scale, dtype, ld=None, ldg=None, off=0, goff=0,
             inplace=False, want_grad=True, stream=None):
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    n, V = x.shape
    ld, ldg = ld or V, ldg or V
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    _, xv = _place(x, ld, off, dt)
    if inplace:
        gv, ldg, gbuf = xv, ld, None
    elif want_grad:
        gbuf, gv = _place(np.full((n, V), 7.0, np.float32), ldg, goff, dt, fill=3.0)
    else:
        gv = None
    loss, margin = (torch.full((npairs,), 9.0, device="cuda") for _ in range(2))
    seq = torch.full((2 * npairs,), 9.0, device="cuda")
    mean, err = torch.full((1,), 9.0, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    nb = vl.vl_preference_workspace_bytes(n, npairs)
    ws = torch.full((nb + 64,), 0xFF, dtype=torch.uint8, device="cuda")       # NaN patterns: nothing is assumed of it
    f = vl.vl_preference_loss_bf16 if dtype == "bf16" else vl.vl_preference_loss
    dev = [H.dev(lab), H.dev(w), H.dev(np.asarray(start, np.int64)), None if ref is None else H.dev(ref)]
    torch.cuda.synchronize()
    f(xv.data_ptr(), ld, n, V, dev[0], dev[1], dev[2], npairs, dev[3], beta, smooth, kind, scale,
      None if gv is None else gv.data_ptr(), ldg, loss, margin, seq, mean, err, workspace=(ws.data_ptr(), nb), stream=stream)
    torch.cuda.synchronize()
    assert bool((ws[nb:] == 0xFF).all())
    if gv is not None and not inplace:
        assert bool((gbuf[:goff] == 3).all()) and bool((gv[:, V:] == 3).all()) and bool((gbuf[goff + n * ldg:] == 3).all())
    return dict(loss=H.host(loss), margin=H.host(margin), seq=H.host(seq), mean=float(mean[0]), err=int(err[0]),
                grad=None if gv is None else _wide(gv, V))


def check_pref(got, x, lab, w, start, npairs, ref, beta, smooth, kind, scale, dtype):
    x = x.astype(np.float64)
    n, V = x.shape
    beta, smooth, scale = (float(np.float32(v)) for v in (beta, smooth, scale))
    want = O.preference(x, lab, w, start, npairs, ref, beta, smooth, kind, scale)
    d = _delta(x, lab, w)
    dlp = np.abs(w) * (d + U * np.abs(want["logp"]))
    tol_s = np.zeros(2 * npairs)
    for s in range(2 * npairs):
        a = min(max(int(start[s]), 0), n)
        tol_s[s] = dlp[a:min(max(int(start[s + 1]), a), n)].sum()
    tol_gap = tol_s[:npairs] + tol_s[npairs:]
    _check(got["seq"], want["seq"], tol_s + 2 * H.EPS * np.abs(np.nan_to_num(want["seq"])), "seq")
    h = np.nan_to_num(want["margin"])
    _check(got["margin"], want["margin"], beta * tol_gap + 4 * H.EPS * np.abs(h), "margin")
    gap = h / beta
    tol_gap = tol_gap + 4 * H.EPS * np.abs(gap)
    slope, bend = np.zeros(npairs), np.zeros(npairs)
    for i in range(npairs):
        slope[i] = abs(O.pair_loss(gap[i], beta, smooth, kind)[1])
        bend[i] = {0: beta * beta / 4, 1: 2.0, 2: 0.0}[kind]
    loss = np.nan_to_num(want["loss"])
    dl = slope * tol_gap + bend * tol_gap ** 2 + U * (np.abs(loss) + (kind == 0))
    _check(got["loss"], want["loss"], dl, "loss")
    if np.isnan(want["mean"]):
        assert np.isnan(got["mean"])
    else:
        assert abs(got["mean"] - want["mean"]) <= dl.mean() + 1e-6 * abs(want["mean"])
    if got["grad"] is not None:
        tol = np.zeros((n, 1))
        for i in range(npairs):
            for s in (i, npairs + i):
                a = min(max(int(start[s]), 0), n)
                b = min(max(int(start[s + 1]), a), n)
                c = scale * np.abs(w[a:b])
                # the factor's own rounding: of its larger term where it is a difference
                tol[a:b, 0] = c * (bend[i] * tol_gap[i] + 2 * U * slope[i] + U * beta * (kind == 0)) + 1e-6 * c * slope[i]
        check_rounded(got["grad"], want["grad"], tol, dtype, "gradient")


def _pairs(lens, V, seed, dtype):
    torch = H.torch_cuda()
    g = np.random.default_rng(seed)
    n = sum(lens)
    x = torch.from_numpy((g.normal(size=(n, V)) * 2).astype(np.float32)).to(dtype).float().numpy()
    lab = g.integers(0, V, n).astype(np.uint32)
    w = (g.random(n) < 0.8).astype(np.float32) * (0.5 + g.random(n)).astype(np.float32)
    start = np.concatenate([[0], np.cumsum(lens)])
    seq = O.preference(x, lab, w, start, len(lens) // 2, None, 0.1, 0.0, 0, 1.0)["seq"]
    return g, x, lab, w, start, (seq + 2 * g.normal(size=len(lens))).astype(np.float32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind,smooth", [(0, 0.0), (0, 0.1), (1, 0.0), (2, 0.0)])
@pytest.mark.parametrize("lens,V", [([1, 1], 1), ([3, 5], 2), ([2, 1, 4, 0], 33), ([7, 12, 3, 9, 1, 5], 4099), ([2, 3], 32003),
                                    ([1, 1], 128256)])
def test_preference(lens, V, kind, smooth, dtype):
    torch = H.torch_cuda()
    g, x, lab, w, start, ref = _pairs(lens, V, sum(lens) * V + kind, torch.bfloat16 if dtype == "bf16" else torch.float32)
    a = (x, lab, w, start, len(lens) // 2, ref, 0.15, smooth, kind, 0.5, dtype)
    got = run_pref(*a)
    assert got["err"] == 0
    check_pref(got, *a)
    b = (x, lab, w, start, len(lens) // 2, None, 2.0, smooth, kind, 0.5, dtype)      # no reference: saturated losses
    check_pref(run_pref(*b, inplace=True), *b)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,ld,off,ldg,goff", [(1000, 1003, 1, 1003, 1), (1000, 1001, 3, 1005, 2), (33001, 33004, 1, 33008, 3)])
def test_preference_strides(V, ld, off, ldg, goff, dtype):
    torch = H.torch_cuda()
    g, x, lab, w, start, ref = _pairs([3, 2, 4, 1], V, V, torch.bfloat16 if dtype == "bf16" else torch.float32)
    lab[:2] = [0, V - 1]
    a = (x, lab, w, start, 2, ref, 0.1, 0.0, 0, 1.0, dtype)
    check_pref(run_pref(*a, ld=ld, off=off, ldg=ldg, goff=goff), *a)
    check_pref(run_pref(*a, ld=ld, off=off, inplace=True), *a)
    check_pref(run_pref(*a, ld=ld, off=off, want_grad=False), *a)


def test_preference_masks_gaps_and_bad_labels():
    torch = H.torch_cuda()
    V = 700
    g, x, lab, w, start, ref = _pairs([4, 3, 5, 2, 6, 4], V, 11, torch.float32)
    n = len(lab)
    # rows before the first and after the last sequence, and a sequence that is masked away whole
    start = start.copy()
    start[0], start[-1] = 2, n - 1
    w[start[1]:start[2]] = 0
    x[start[1]] = np.nan
    w[[0, 1, n - 1]] = 1.0
    a = (x, lab, w, start, 3, ref, 0.1, 0.0, 0, 1.0, "f32")
    got = run_pref(*a)
    assert got["err"] == 0 and not got["grad"][[0, 1, n - 1]].any() and got["seq"][1] == 0
    check_pref(got, *a)
    # a bad label takes its pair out, and only that one; a bad label outside every sequence changes nothing
    lab2 = lab.copy()
    t = start[3]
    w[t] = 1.0
    lab2[t], lab2[0] = V, 0xFFFFFFFF
    a = (x, lab2, w, start, 3, ref, 0.1, 0.0, 0, 1.0, "f32")
    got = run_pref(*a)
    assert got["err"] == 2 and np.isnan(got["loss"][0]) and np.isnan(got["seq"][3]) and np.isnan(got["mean"])
    assert not got["grad"][start[3]:start[4]].any() and not got["grad"][start[0]:start[1]].any() and not got["grad"][0].any()
    for k in ("loss", "margin"):
        assert np.isfinite(got[k][1:]).all()
    check_pref(got, *a)
    # everything masked: ln 2 each against a zero reference, no gradient
    z = run_pref(x, lab, np.zeros(n, np.float32), start, 3, None, 0.1, 0.0, 0, 1.0, "f32")
    assert np.allclose(z["loss"], np.log(2)) and not z["grad"].any() and not z["seq"].any()
    # starts outside the rows are clamped, never followed
    wild = np.array([-5, 3, 1 << 40, 4, 6, 1 << 62, n + 9], np.int64)
    assert np.isfinite(run_pref(x, lab, w * 0 + 1e-3 * (np.arange(n) != start[1]).astype(np.float32), wild, 3, ref, 0.1, 0.0,
                                0, 1.0, "f32")["loss"]).all()


def test_preference_many_rows_and_streams():
    torch = H.torch_cuda()
    g = np.random.default_rng(0)
    lens = list(g.integers(1, 40, 60))
    g, x, lab, w, start, ref = _pairs(lens, 2100, 21, torch.bfloat16)
    a = (x, lab, w, start, 30, ref, 0.1, 0.1, 0, 1 / 30, "bf16")
    p = run_pref(*a, stream=torch.cuda.Stream())
    check_pref(p, *a)
    q = run_pref(*a, inplace=True)
    assert np.array_equal(p["grad"], q["grad"]) and np.array_equal(p["loss"], q["loss"]) and p["mean"] == q["mean"]


def test_gradients_against_differences_of_the_losses():
    """A step along the gradient changes the kernels' own losses by the gradient's square."""
    torch = H.torch_cuda()
    g, x, act, old, ref = _inputs(6, 50, 31, torch.float32)
    adv, w = g.normal(size=6).astype(np.float32), np.full(6, 1.0, np.float32)
    a = (act, old, ref, adv, w, 0.1, 1.0, "f32")
    o = run_policy(x, *a)
    h = 1e-2
    up = run_policy((x + h * o["grad"]).astype(np.float32), *a)["total"]
    dn = run_policy((x - h * o["grad"]).astype(np.float32), *a)["total"]
    n2 = (o["grad"] ** 2).sum()
    assert abs((up - dn) / (2 * h) - n2) < 2e-3 * n2
    g, x, lab, w, start, ref = _pairs([4, 3, 2, 5], 60, 5, torch.float32)
    for kind in (0, 1):
        b = (lab, w, start, 2, ref, 0.2, 0.1, kind, 0.5, "f32")
        o = run_pref(x, *b)
        n2 = (o["grad"] ** 2).sum()
        h = 1e-2 / max(1.0, n2 ** 0.5)
        up = run_pref((x + h * o["grad"]).astype(np.float32), *b)["mean"]
        dn = run_pref((x - h * o["grad"]).astype(np.float32), *b)["mean"]
        assert abs((up - dn) / (2 * h) - n2) < 1e-2 * n2
