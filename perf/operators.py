"""The post-training operators of the vocabulary head, in cases that can be timed and compared.

    policy   the clipped policy loss with a KL term over rows of logits: losses, log-probabilities,
             KL estimates and the gradient of the logits (vl_policy_loss, fp32 and bf16)
    pref     the preference loss over pairs of sequences (paired log ratios): losses, margins,
             sequence log-probabilities and the gradient of the logits (vl_preference_loss)
    norm     the layer norm before the head, forward (vl_layernorm_fwd) or forward and backward
             with the weight's and the bias's gradient (vl_layernorm_bwd)
    fp8      the head's product in 8-bit floating point: hidden rows quantised with a scale for
             each 128 columns, times a weight plane with a scale for each 128 x 128 block
             (vl_quant_fp8_rows, vl_gemm_fp8_tn)

``run`` computes an operator in plain torch in 32 bits (``own`` false), or calls the library's
entry points (``own`` true).  ``exact`` computes the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

# ---------------------------------------------------------------- cases


def listed():
    return [
        # the last tokens of one short response, small test vocabulary: launch latency
        dict(name="policy_tiny", op="policy", dtype="f32", ntok=64, V=1024, seqs=1, prompt=8, kl=0.04),
        # one training micro-batch of a 32000-word model, logits kept in bf16
        dict(name="policy_lm_bf16", op="policy", dtype="bf16", ntok=2048, V=32000, seqs=8, prompt=64, kl=0.02),
        # a vocabulary padded to nothing: every row starts at another alignment; no reference model
        dict(name="policy_ragged", op="policy", dtype="f32", ntok=1021, V=32003, seqs=3, prompt=41, kl=0.0),
        # a large vocabulary's micro-batch, fp32 logits
        dict(name="policy_large", op="policy", dtype="f32", ntok=4096, V=128256, seqs=8, prompt=64, kl=0.04),
        # two pairs of a few tokens: launch latency
        dict(name="pref_tiny", op="pref", dtype="f32", pairs=2, longest=24, prompt=4, V=1024, kind="sigmoid", smooth=0.0),
        # a micro-batch of pairs of unequal lengths with a smoothed label
        dict(name="pref_lm", op="pref", dtype="f32", pairs=8, longest=129, prompt=17, V=32000, kind="sigmoid", smooth=0.1),
        # long pairs over a large vocabulary, bf16 logits, the squared form
        dict(name="pref_large_bf16", op="pref", dtype="bf16", pairs=8, longest=256, prompt=32, V=128256, kind="ipo", smooth=0.0),
        # a decoding step's rows before the head: launch latency
        dict(name="norm_decode", op="norm", dtype="bf16", rows=8, hs=4096, back=False, dy="bf16"),
        # training rows forward and backward; the head hands its gradient back in fp32
        dict(name="norm_train", op="norm", dtype="bf16", rows=16384, hs=4096, back=True, dy="f32"),
        # an odd hidden size, fp32 throughout
        dict(name="norm_ragged", op="norm", dtype="f32", rows=3001, hs=2050, back=True, dy="f32"),
        # a decoding step's logits: the weight plane is what has to be read
        dict(name="fp8_decode", op="fp8", rows=8, V=32000, hs=4096),
        # scoring a chunk of rows with a frozen model: tensor-core work
        dict(name="fp8_head", op="fp8", rows=2048, V=128256, hs=4096),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["policy", "pref", "norm", "fp8"])
    if op == "policy":
        V = _log_int(rng, 1000, 131072)
        ntok = _log_int(rng, 32, min(8192, 4096 * 128256 // V))
        seqs = rng.randint(1, 8)
        return dict(op=op, dtype=rng.choice(["f32", "bf16"]), ntok=ntok, V=V, seqs=seqs,
                    prompt=rng.randint(0, ntok // (4 * seqs)), kl=rng.choice([0.0, 0.04]))
    if op == "pref":
        V = _log_int(rng, 1000, 131072)
        pairs = _log_int(rng, 1, 32)
        longest = _log_int(rng, 8, max(8, min(512, 4096 * 128256 // (2 * pairs * V))))
        return dict(op=op, dtype=rng.choice(["f32", "bf16"]), pairs=pairs, longest=longest,
                    prompt=rng.randint(0, longest // 4), V=V, kind=rng.choice(["sigmoid", "ipo"]),
                    smooth=rng.choice([0.0, 0.1]))
    if op == "norm":
        hs = _log_int(rng, 256, 12288)
        rows = _log_int(rng, 1, min(32768, 16384 * 8192 // hs))
        dtype = rng.choice(["f32", "bf16"])
        return dict(op=op, dtype=dtype, rows=rows, hs=hs, back=rng.random() < 0.6,
                    dy="f32" if dtype == "f32" else rng.choice(["f32", "bf16"]))
    V = _log_int(rng, 1000, 131072)
    return dict(op=op, rows=_log_int(rng, 1, 2048), V=V, hs=16 * _log_int(rng, 16, 256))


# ---------------------------------------------------------------- inputs


def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _pref_lengths(case):
    """Token counts of the 2 pairs sequences: chosen 0 .. pairs-1, then rejected, unequal."""
    n, longest = case["pairs"], case["longest"]
    floor = max(case["prompt"] + 1, longest // 2)
    return [max(floor, longest - (5 * s) % (longest // 2 + 1)) for s in range(2 * n)]


def _logits(g, ntok, V, dtype, picked):
    """N(0, 3^2) logits, three rows in ten with the picked column raised by 8 (a confident model)."""
    x = torch.randn(ntok, V, device="cuda", generator=g).mul_(3.0)
    sure = (torch.rand(ntok, device="cuda", generator=g) < 0.3).float() * 8.0
    x.scatter_add_(1, picked[:, None], sure[:, None])
    return x.to(dtype)


def _logp32(x, picked):
    """Log-probabilities of the picked columns, a block of rows at a time."""
    out = torch.empty(x.shape[0], device="cuda")
    for a in range(0, x.shape[0], 1024):
        out[a:a + 1024] = torch.log_softmax(x[a:a + 1024].float(), 1).gather(1, picked[a:a + 1024, None])[:, 0]
    return out


def _by_sequence(v, of, n):
    """Sums of v over the tokens of each sequence, in a fixed order."""
    return torch.where(of == torch.arange(n, device=v.device)[:, None], v, torch.zeros_like(v)).sum(1)


CLIP_LO, CLIP_HI = 0.2, 0.28


def _prepare_policy(case, g):
    ntok, V, seqs = case["ntok"], case["V"], case["seqs"]
    dt = _dt(case["dtype"])
    act = torch.randint(0, V, (ntok,), device="cuda", generator=g)
    x = _logits(g, ntok, V, dt, act)
    logp = _logp32(x, act)
    # the sampler's log-probabilities: a few updates old; kept off the two clip edges, where the
    # gradient jumps and two roundings of the same ratio may land on different sides
    d = 0.25 * torch.randn(ntok, device="cuda", generator=g)
    for edge in (math.log(1 - CLIP_LO), math.log(1 + CLIP_HI)):
        near = (d - edge).abs() < 4e-3
        d = torch.where(near, d + torch.where(d < edge, -8e-3, 8e-3), d)
    of = torch.arange(ntok, device="cuda") * seqs // ntok
    first = torch.searchsorted(of, torch.arange(seqs, device="cuda"))
    at = torch.arange(ntok, device="cuda") - first[of]
    live = at >= case["prompt"]
    return dict(case=case, x=x, act=act.to(torch.int32), act64=act, old=logp - d,
                ref=logp + 0.3 * torch.randn(ntok, device="cuda", generator=g) if case["kl"] else None,
                adv=torch.randn(seqs, device="cuda", generator=g)[of].contiguous(),
                weight=live.float() / live.sum().clamp(min=1),
                grad=torch.empty_like(x), loss=torch.empty(ntok, device="cuda"),
                logp=torch.empty(ntok, device="cuda"), kl=torch.empty(ntok, device="cuda"),
                total=torch.empty(1, device="cuda"))


def _prepare_pref(case, g):
    lens = _pref_lengths(case)
    n, V, dt = case["pairs"], case["V"], _dt(case["dtype"])
    ntok = sum(lens)
    start = torch.tensor([0] + lens).cumsum(0).cuda()
    lab = torch.randint(0, V, (ntok,), device="cuda", generator=g)
    x = _logits(g, ntok, V, dt, lab)
    of = torch.repeat_interleave(torch.arange(2 * n, device="cuda"), torch.tensor(lens, device="cuda"))
    at = torch.arange(ntok, device="cuda") - start[of]
    weight = (at >= case["prompt"]).float()
    if case["kind"] == "ipo":       # the squared form is taken over the mean log-probability of a sequence
        weight = weight / torch.tensor([m - case["prompt"] for m in lens], device="cuda").float()[of]
    seq = _by_sequence((weight * _logp32(x, lab)).double(), of, 2 * n)
    drift = 3.0 if case["kind"] == "sigmoid" else 0.5
    ref = seq + drift * torch.randn(2 * n, device="cuda", generator=g, dtype=torch.float64)
    need = 0
    if own:
        from top_kl_distill_gb300 import vloss as vl
        need = vl.vl_preference_workspace_bytes(ntok, n)
    return dict(case=case, x=x, lab=lab.to(torch.int32), lab64=lab, start=start, of=of, weight=weight, ref=ref.float(),
                ntok=ntok, grad=torch.empty_like(x), loss=torch.empty(n, device="cuda"),
                margin=torch.empty(n, device="cuda"), seq=torch.empty(2 * n, device="cuda"),
                mean=torch.empty(1, device="cuda"), ws=torch.empty(max(16, need), dtype=torch.uint8, device="cuda"))


def _prepare_norm(case, g):
    rows, hs, dt = case["rows"], case["hs"], _dt(case["dtype"])
    spread = torch.exp(0.5 * torch.randn(hs, device="cuda", generator=g))      # channels of unequal size
    x = torch.randn(rows, hs, device="cuda", generator=g).mul_(spread).add_(0.25).to(dt)
    s = dict(case=case, x=x, gamma=1 + 0.2 * torch.randn(hs, device="cuda", generator=g),
             beta=0.1 * torch.randn(hs, device="cuda", generator=g), y=torch.empty_like(x),
             mu=torch.empty(rows, device="cuda"), rstd=torch.empty(rows, device="cuda"))
    if case["back"]:
        need = 0
        if own:
            from top_kl_distill_gb300 import vloss as vl
            need = vl.vl_layernorm_bwd_workspace_bytes(rows, hs)
        s.update(dy=(torch.randn(rows, hs, device="cuda", generator=g) / rows).to(_dt(case["dy"])),
                 dx=torch.empty_like(x), dgamma=torch.empty(hs, device="cuda"), dbeta=torch.empty(hs, device="cuda"),
                 ws=torch.empty(max(16, need), dtype=torch.uint8, device="cuda"))
    return s


BLK = 128
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100       # the least amax a scale is made from, so that an empty block has one too


def _up(n, m):
    return -(-n // m)


def _prepare_fp8(case, g):
    m, n, k = case["rows"], case["V"], case["hs"]
    x = torch.randn(m, k, device="cuda", generator=g)
    x[:, torch.randint(0, k, (max(1, k // 256),), device="cuda", generator=g)] *= 20.0     # outlier channels
    w = torch.randn(n, k, device="cuda", generator=g).div_(math.sqrt(k)).to(torch.bfloat16)
    nb, kb = _up(n, BLK), _up(k, BLK)
    wq = torch.empty(n, k, dtype=torch.uint8, device="cuda")
    ws = torch.empty(nb, kb, device="cuda")
    for b in range(nb):            # the weight plane is quantised once, when a program loads it
        r = w[b * BLK:(b + 1) * BLK].float()
        r = torch.nn.functional.pad(r, (0, kb * BLK - k)).view(-1, kb, BLK)
        ws[b] = r.abs().amax((0, 2)).clamp(min=AMAX_FLOOR) / E4M3_MAX
        q = (r / ws[b][None, :, None]).reshape(-1, kb * BLK)[:, :k]
        wq[b * BLK:(b + 1) * BLK] = q.to(torch.float8_e4m3fn).view(torch.uint8)
    return dict(case=case, x=x.to(torch.bfloat16), wq=wq, ws=ws, q=torch.empty(m, k, dtype=torch.uint8, device="cuda"),
                qs=torch.empty(kb, m, device="cuda"), y=torch.empty(m, n, device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    return {"policy": _prepare_policy, "pref": _prepare_pref, "norm": _prepare_norm, "fp8": _prepare_fp8}[case["op"]](case, g)


# ---------------------------------------------------------------- the library's calls


KINDS = {"sigmoid": 0, "ipo": 1, "hinge": 2}
PREF_BETA = 0.1


def _own(s):
    from top_kl_distill_gb300 import vloss as vl
    c = s["case"]
    if c["op"] == "policy":
        f = vl.vl_policy_loss_bf16 if c["dtype"] == "bf16" else vl.vl_policy_loss
        f(s["x"], c["V"], c["ntok"], c["V"], s["act"], s["old"], s["ref"], s["adv"], s["weight"], CLIP_LO, CLIP_HI,
          c["kl"], 1.0, s["grad"], c["V"], s["loss"], s["logp"], s["kl"], s["total"])
        return [s["grad"], s["loss"], s["logp"], s["kl"], s["total"]]
    if c["op"] == "pref":
        f = vl.vl_preference_loss_bf16 if c["dtype"] == "bf16" else vl.vl_preference_loss
        f(s["x"], c["V"], s["ntok"], c["V"], s["lab"], s["weight"], s["start"], c["pairs"], s["ref"], PREF_BETA,
          c["smooth"], KINDS[c["kind"]], 1.0 / c["pairs"], s["grad"], c["V"], s["loss"], s["margin"], s["seq"],
          s["mean"], workspace=s["ws"])
        return [s["grad"], s["loss"], s["margin"], s["seq"], s["mean"]]
    if c["op"] == "norm":
        bf = c["dtype"] == "bf16"
        f = vl.vl_layernorm_fwd_bf16 if bf else vl.vl_layernorm_fwd
        f(s["x"], c["hs"], c["rows"], c["hs"], s["gamma"], s["beta"], 1e-5, s["y"], c["hs"], s["mu"], s["rstd"])
        out = [s["y"], s["mu"], s["rstd"]]
        if c["back"]:
            f = vl.vl_layernorm_bwd_bf16 if bf else vl.vl_layernorm_bwd
            f(s["dy"], c["hs"], s["x"], c["hs"], c["rows"], c["hs"], s["gamma"], s["mu"], s["rstd"], s["dx"], c["hs"],
              s["dgamma"], s["dbeta"], workspace=s["ws"])
            out += [s["dx"], s["dgamma"], s["dbeta"]]
        return out
    m, n, k = c["rows"], c["V"], c["hs"]
    vl.vl_quant_fp8_rows_bf16(s["x"], k, m, k, s["q"], s["qs"])
    vl.vl_gemm_fp8_tn(s["q"], s["qs"], s["wq"], s["ws"], s["y"], m, n, k, n)
    return [s["y"]]


# ---------------------------------------------------------------- plain forms, 32 bits


def _softmax_logp(x, picked):
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - m)
    z = e.sum(1, keepdim=True)
    return e / z, ((x.gather(1, picked[:, None]) - m) - torch.log(z))[:, 0]


def _row_grad(p, picked, dlogp):
    """dlogp * (onehot - softmax) of each row."""
    gr = p.mul_(-dlogp[:, None])
    gr.scatter_add_(1, picked[:, None], dlogp[:, None])
    return gr


def _plain_policy(s):
    c = s["case"]
    p, logp = _softmax_logp(s["x"].float(), s["act64"])
    live = s["weight"] != 0
    ratio = torch.exp(logp - s["old"])
    adv = s["adv"]
    free, held = ratio * adv, ratio.clamp(1 - CLIP_LO, 1 + CLIP_HI) * adv
    each = -torch.minimum(free, held)
    dlogp = torch.where(free <= held, -ratio * adv, torch.zeros_like(adv))
    kl = torch.zeros_like(logp)
    if s["ref"] is not None:
        d = s["ref"] - logp
        kl = torch.exp(d) - d - 1
        each = each + c["kl"] * kl
        dlogp = dlogp + c["kl"] * (1 - torch.exp(d))
    zero = torch.zeros_like(logp)
    loss = torch.where(live, s["weight"] * each, zero)
    dlogp = torch.where(live, s["weight"] * dlogp, zero)
    return [_row_grad(p, s["act64"], dlogp).to(s["x"].dtype), loss, torch.where(live, logp, zero),
            torch.where(live, kl, zero), loss.sum()[None]]


def _plain_pref(s):
    c, n = s["case"], s["case"]["pairs"]
    p, logp = _softmax_logp(s["x"].float(), s["lab64"])
    seq = _by_sequence(torch.where(s["weight"] != 0, s["weight"] * logp, torch.zeros_like(logp)), s["of"], 2 * n)
    gap = (seq - s["ref"])[:n] - (seq - s["ref"])[n:]
    if c["kind"] == "sigmoid":
        h = PREF_BETA * gap
        def soft(v):                                      # ln(1 + e^v)
            return v.clamp(min=0) + torch.log(1 + torch.exp(-v.abs()))
        loss = (1 - c["smooth"]) * soft(-h) + c["smooth"] * soft(h)
        dgap = PREF_BETA * (c["smooth"] - 1 / (1 + torch.exp(h)))
    else:
        d = gap - 0.5 / PREF_BETA
        loss, dgap = d * d, 2 * d
    side = torch.cat([dgap, -dgap]) / n
    dlogp = torch.where(s["weight"] != 0, s["weight"] * side[s["of"]], torch.zeros_like(logp))
    return [_row_grad(p, s["lab64"], dlogp).to(s["x"].dtype), loss, PREF_BETA * gap, seq, loss.mean()[None]]


def _plain_norm(s):
    x = s["x"].float()
    mu = x.mean(1, keepdim=True)
    xc = x - mu
    rstd = 1 / torch.sqrt((xc * xc).mean(1, keepdim=True) + 1e-5)
    xh = xc * rstd
    out = [(xh * s["gamma"] + s["beta"]).to(s["x"].dtype), mu[:, 0], rstd[:, 0]]
    if s["case"]["back"]:
        dy = s["dy"].float()
        t = dy * s["gamma"]
        dx = rstd * (t - t.mean(1, keepdim=True) - xh * (t * xh).mean(1, keepdim=True))
        out += [dx.to(s["x"].dtype), (dy * xh).sum(0), dy.sum(0)]
    return out


def _plain_fp8(s):
    m, k = s["case"]["rows"], s["case"]["hs"]
    kb = _up(k, BLK)
    x = torch.nn.functional.pad(s["x"].float(), (0, kb * BLK - k)).view(m, kb, BLK)
    sc = x.abs().amax(2).clamp(min=AMAX_FLOOR) / E4M3_MAX
    x = (x / sc[:, :, None]).to(torch.float8_e4m3fn).float() * sc[:, :, None]
    x = x.view(m, kb * BLK)[:, :k]
    w = s["wq"].view(torch.float8_e4m3fn).float()
    w *= s["ws"].repeat_interleave(BLK, 0)[:w.shape[0]].repeat_interleave(BLK, 1)[:, :k]
    return [x @ w.t()]


def run(state):
    if own:
        return _own(state)
    return {"policy": _plain_policy, "pref": _plain_pref, "norm": _plain_norm, "fp8": _plain_fp8}[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    op = case["op"]
    es = 2 if case.get("dtype") == "bf16" else 4
    if op == "policy":
        n, V = case["ntok"], case["V"]
        starts = [-(-s * n // case["seqs"]) for s in range(case["seqs"] + 1)]
        live = sum(max(0, b - a - case["prompt"]) for a, b in zip(starts, starts[1:]))
        # a live row is read once; every row's gradient is written once
        return {"bytes": (live + n) * V * es + n * 4 * (8 if case["kl"] else 7), "flops": 6 * live * V}
    if op == "pref":
        lens, V = _pref_lengths(case), case["V"]
        live = sum(m - case["prompt"] for m in lens)
        return {"bytes": (live + sum(lens)) * V * es + sum(lens) * 8 + case["pairs"] * 40, "flops": 6 * live * V}
    if op == "norm":
        rows, hs = case["rows"], case["hs"]
        b = 2 * rows * hs * es + 8 * hs + 8 * rows
        f = 8 * rows * hs
        if case["back"]:           # x is there already from the forward pass, but no cache holds it at size
            b += rows * hs * (2 * es + (2 if case["dy"] == "bf16" else 4)) + 12 * hs + 8 * rows
            f += 14 * rows * hs
        return {"bytes": b, "flops": f}
    m, n, k = case["rows"], case["V"], case["hs"]
    return {"bytes": 2 * m * k + n * k + 4 * _up(n, BLK) * _up(k, BLK) + 4 * m * n, "flops": 2 * m * n * k}


# ---------------------------------------------------------------- the definitions in 64 bits


def _exact_rows(x, picked, live):
    """log softmax(x)[picked] of the live rows in 64 bits, 0 elsewhere."""
    out = torch.zeros(x.shape[0], dtype=torch.float64, device=x.device)
    for a in range(0, x.shape[0], 512):
        b = x[a:a + 512].double()
        v = b[torch.arange(b.shape[0], device=x.device), picked[a:a + 512]] - torch.logsumexp(b, 1)
        out[a:a + 512] = torch.where(live[a:a + 512], v, torch.zeros_like(v))
    return out


def _exact_grad(x, picked, dlogp):
    """d(sum dlogp_t logp_t)/dx in 64 bits."""
    gr = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for a in range(0, x.shape[0], 512):
        b = torch.softmax(x[a:a + 512].double(), 1).neg_()
        b[torch.arange(b.shape[0], device=x.device), picked[a:a + 512]] += 1.0
        gr[a:a + 512] = b * dlogp[a:a + 512, None]
    return gr


def _e4m3(v):
    """The nearest e4m3 value of each |v| <= 448 (ties to even), by the spacing of its binade."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=-6) - 3)
    return torch.round(v / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "policy":
        w, adv = s["weight"].double(), s["adv"].double()
        live = s["weight"] != 0
        logp = _exact_rows(s["x"], s["act64"], live)
        r = (logp - s["old"].double()).exp()
        lo, hi = 1 - float(torch.tensor(CLIP_LO)), 1 + float(torch.tensor(CLIP_HI))
        capped = torch.where(adv >= 0, r.clamp(max=hi), r.clamp(min=lo))
        obj, dobj = capped * adv, torch.where(capped == r, r * adv, torch.zeros_like(r))
        kl, dkl = torch.zeros_like(r), torch.zeros_like(r)
        if s["ref"] is not None:
            q = (s["ref"].double() - logp)
            kl, dkl = torch.expm1(q) - q, -torch.expm1(q)
        beta = float(torch.tensor(case["kl"]))
        loss = torch.where(live, w * (beta * kl - obj), torch.zeros_like(w))
        d = torch.where(live, w * (beta * dkl - dobj), torch.zeros_like(w))
        return [_exact_grad(s["x"], s["act64"], d), loss, logp, torch.where(live, kl, torch.zeros_like(kl)), loss.sum()[None]]
    if op == "pref":
        n, w = case["pairs"], s["weight"].double()
        logp = _exact_rows(s["x"], s["lab64"], s["weight"] != 0)
        ends = s["start"].tolist()
        seq = torch.stack([(w[a:b] * logp[a:b]).sum() for a, b in zip(ends, ends[1:])])
        lift = seq - s["ref"].double()
        beta, eps = float(torch.tensor(PREF_BETA)), float(torch.tensor(case["smooth"]))
        gap = lift[:n] - lift[n:]
        if case["kind"] == "sigmoid":
            ls = torch.nn.functional.logsigmoid
            loss = -(1 - eps) * ls(beta * gap) - eps * ls(-beta * gap)
            dgap = beta * (eps * torch.sigmoid(beta * gap) - (1 - eps) * torch.sigmoid(-beta * gap))
        else:
            loss, dgap = (gap - 1 / (2 * beta)) ** 2, 2 * (gap - 1 / (2 * beta))
        d = torch.zeros_like(w)
        for i in range(2 * n):
            d[ends[i]:ends[i + 1]] = w[ends[i]:ends[i + 1]] * (dgap[i] if i < n else -dgap[i - n]) / n
        return [_exact_grad(s["x"], s["lab64"], d), loss, beta * gap, seq, loss.mean()[None]]
    if op == "norm":
        x, ga = s["x"].double(), s["gamma"].double()
        var, mu = torch.var_mean(x, 1, correction=0)
        inv = (var + float(torch.tensor(1e-5))).rsqrt()
        hat = (x - mu[:, None]) * inv[:, None]
        out = [hat * ga + s["beta"].double(), mu, inv]
        if case["back"]:
            dy = s["dy"].double()
            u = dy * ga
            a, b = u.sum(1) / case["hs"], (u * hat).sum(1) / case["hs"]
            out += [(u - a[:, None] - b[:, None] * hat) * inv[:, None], torch.einsum("rc,rc->c", dy, hat), dy.sum(0)]
        return out
    m, n, k = case["rows"], case["V"], case["hs"]
    x = s["x"].float()
    y = torch.zeros(m, n, dtype=torch.float64, device="cuda")
    for b in range(_up(k, BLK)):       # block by block of the contraction
        xb = x[:, b * BLK:(b + 1) * BLK]
        sx = torch.maximum(xb.abs().max(1).values, torch.tensor(AMAX_FLOOR, device="cuda")) / E4M3_MAX
        xq = _e4m3(xb / sx[:, None]).double() * sx.double()[:, None]
        wb = s["wq"][:, b * BLK:(b + 1) * BLK].contiguous().view(torch.float8_e4m3fn).double()
        y += xq @ (wb * s["ws"][:, b].double().repeat_interleave(BLK)[:n, None]).t()
    return [y]
