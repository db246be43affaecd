"""Plain float64 definitions of the post-training operators, one row or pair at a time.

Test infrastructure: only tests and the smoke check import it.  Inputs are the values the
kernels get (fp32, or bf16 widened), outputs float64.
"""
from __future__ import annotations

import math

import numpy as np


def row_logp(x, a):
    """(logp of column a, softmax) of one row."""
    x = np.asarray(x, np.float64)
    m = x.max()
    e = np.exp(x - m)
    z = e.sum()
    return (x[a] - m) - math.log(z), e / z


def policy(x, act, old, ref, adv, weight, clip_lo, clip_hi, kl_coef, scale):
    """Per-row loss, logp, kl, factor G and the gradient; rows of weight 0 are not read."""
    n, V = x.shape
    loss, logp, kl, G = np.zeros(n), np.zeros(n), np.zeros(n), np.zeros(n)
    grad = np.zeros((n, V))
    for t in range(n):
        w = float(weight[t])
        if w == 0:
            continue
        if act[t] >= V:
            loss[t] = logp[t] = np.nan
            continue
        lp, p = row_logp(x[t], act[t])
        r = np.exp(lp - float(old[t]))
        A = float(adv[t])
        free, held = r * A, min(max(r, 1 - float(clip_lo)), 1 + float(clip_hi)) * A
        each = -min(free, held)
        d = -r * A if free <= held else 0.0
        if ref is not None:
            q = float(ref[t]) - lp
            kl[t] = math.expm1(q) - q if q < 700 else np.inf
            if kl_coef:
                each += kl_coef * kl[t]
                d -= kl_coef * (math.expm1(q) if q < 700 else np.inf)
        loss[t], logp[t], G[t] = w * each, lp, w * d
        if scale * G[t] != 0:
            one = np.zeros(V)
            one[act[t]] = 1.0
            grad[t] = scale * G[t] * (one - p)
    return dict(loss=loss, logp=logp, kl=kl, G=G, grad=grad, total=loss.sum())


def pair_loss(gap, beta, smooth, kind):
    """(loss, d loss / d gap) of one pair; kind 0 sigmoid, 1 squared, 2 hinge."""
    if kind == 0:
        h = beta * gap
        def sp(v):
            return max(v, 0.0) + math.log1p(math.exp(-abs(v)))
        sg = 1 / (1 + math.exp(-h)) if h >= 0 else math.exp(h) / (1 + math.exp(h))
        sn = 1 / (1 + math.exp(h)) if h <= 0 else math.exp(-h) / (1 + math.exp(-h))
        return (1 - smooth) * sp(-h) + smooth * sp(h), beta * (smooth * sg - (1 - smooth) * sn)
    if kind == 1:
        d = gap - 1 / (2 * beta)
        return d * d, 2 * d
    h = beta * gap
    return (1 - h, -beta) if h < 1 else (0.0, 0.0)


def preference(x, lab, weight, start, npairs, ref, beta, smooth, kind, scale):
    n, V = x.shape
    logp, bad = np.zeros(n), np.zeros(n, bool)
    for t in range(n):
        if weight[t] != 0:
            if lab[t] >= V:
                bad[t] = True
            else:
                logp[t] = row_logp(x[t], lab[t])[0]
    seq = np.zeros(2 * npairs)
    rows = []
    for s in range(2 * npairs):
        a = min(max(int(start[s]), 0), n)
        b = min(max(int(start[s + 1]), a), n)
        rows.append((a, b))
        seq[s] = np.nan if bad[a:b].any() else sum(float(weight[t]) * logp[t] for t in range(a, b) if weight[t] != 0)
    loss, margin, grad = np.zeros(npairs), np.zeros(npairs), np.zeros((n, V))
    for i in range(npairs):
        rc, rr = (0.0, 0.0) if ref is None else (float(ref[i]), float(ref[npairs + i]))
        gap = (seq[i] - rc) - (seq[npairs + i] - rr)
        if np.isnan(gap):
            loss[i] = margin[i] = np.nan
            continue
        margin[i] = beta * gap
        loss[i], d = pair_loss(gap, beta, smooth, kind)
        for s, sign in ((i, 1.0), (npairs + i, -1.0)):
            for t in range(*rows[s]):
                c = scale * sign * d * float(weight[t])
                if c != 0:
                    one = np.zeros(V)
                    one[lab[t]] = 1.0
                    grad[t] = c * (one - row_logp(x[t], lab[t])[1])
    return dict(loss=loss, margin=margin, seq=seq, grad=grad, mean=loss.mean() if npairs else 0.0, logp=logp)


def layernorm(x, gamma, beta, eps):
    x = np.asarray(x, np.float64)
    mu = x.mean(1)
    rstd = 1 / np.sqrt(((x - mu[:, None]) ** 2).mean(1) + float(eps))
    return ((x - mu[:, None]) * rstd[:, None]) * gamma + beta, mu, rstd


def layernorm_bwd(dy, x, gamma, mu, rstd):
    """dx, dgamma, dbeta from the statistics as given."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    xh = (x - np.asarray(mu, np.float64)[:, None]) * np.asarray(rstd, np.float64)[:, None]
    t = dy * gamma
    dx = np.asarray(rstd, np.float64)[:, None] * (t - t.mean(1, keepdims=True) - xh * (t * xh).mean(1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


# ---------------------------------------------------------------- e4m3

_TABLE = np.array([(-1.0 if b & 0x80 else 1.0) *
                   ((b & 7) * 2.0 ** -9 if (b >> 3) & 15 == 0 else (8 + (b & 7)) * 2.0 ** (((b >> 3) & 15) - 10))
                   for b in range(256)])
_TABLE[0x7F] = _TABLE[0xFF] = np.nan
_POS = _TABLE[:0x7F]
_INV448 = np.float32(1) / np.float32(448)


def e4m3_value(b):
    return _TABLE[np.asarray(b)]


def e4m3_byte(v):
    """The byte of the nearest e4m3 value, ties to the even byte, saturating; NaN to 0x7F (sign kept)."""
    v = np.asarray(v, np.float64)
    a = np.minimum(np.abs(v), 448.0)
    hi = np.clip(np.searchsorted(_POS, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    pick = np.where(_POS[hi] == a, hi, pick)
    pick = np.where(np.isnan(v), 0x7F, pick)
    return (pick | np.where(np.signbit(v), 0x80, 0)).astype(np.uint8)


def quant_rows(x):
    """(bytes [M][K], scales [ceil(K/128)][M]) of fp32 rows: scale = amax * fp32(1/448) and
    x / scale, each rounded to fp32, then to e4m3."""
    x = np.asarray(x, np.float32)
    M, K = x.shape
    kb = -(-K // 128)
    q, s = np.zeros((M, K), np.uint8), np.zeros((kb, M), np.float32)
    for b in range(kb):
        blk = x[:, b * 128:(b + 1) * 128]
        amax = np.fmax.reduce(np.abs(blk), axis=1)
        s[b] = np.fmax(amax, np.float32(2.0 ** -100)) * _INV448
        with np.errstate(invalid="ignore"):
            q[:, b * 128:(b + 1) * 128] = e4m3_byte(blk / s[b][:, None])
    return q, s


def quant_blocks(w):
    w = np.asarray(w, np.float32)
    N, K = w.shape
    nb, kb = -(-N // 128), -(-K // 128)
    q, s = np.zeros((N, K), np.uint8), np.zeros((nb, kb), np.float32)
    for i in range(nb):
        for b in range(kb):
            blk = w[i * 128:(i + 1) * 128, b * 128:(b + 1) * 128]
            s[i, b] = max(np.abs(blk).max(), np.float32(2.0 ** -100)) * _INV448
            q[i * 128:(i + 1) * 128, b * 128:(b + 1) * 128] = e4m3_byte(blk / s[i, b])
    return q, s


def gemm_fp8(qa, sa, qb, sb, alpha=1.0):
    """(product, sum of the absolute products) in float64."""
    M, K = qa.shape
    N = qb.shape[0]
    out, mag = np.zeros((M, N)), np.zeros((M, N))
    for b in range(-(-K // 128)):
        c = slice(b * 128, (b + 1) * 128)
        A = e4m3_value(qa[:, c]) * sa[b].astype(np.float64)[:, None]
        B = e4m3_value(qb[:, c]) * np.repeat(sb[:, b].astype(np.float64), 128)[:N, None]
        out += A @ B.T
        mag += np.abs(A) @ np.abs(B).T
    return alpha * out, abs(alpha) * mag
