"""Layer norm forward and backward on the GPU against the float64 definition.

Tolerances, from the arithmetic: a row's sums run over at most 16384 terms, at most 64 in a
row by one thread and then up a tree, so a sum is off by at most 128 * 2^-24 of the sum of its
terms' sizes; the column sums by (rows / 32 + 64) * 2^-24 of theirs.  Elementwise steps add a few
2^-24 of the terms.  bf16 outputs lie between the bf16 roundings of the fp32 interval's ends.
"""
import numpy as np
import pytest

from oracle import post_oracle as O
from tests import gpu_harness as H
from tests.test_gpu_post_loss import _check, _place, _wide, check_rounded

pytestmark = pytest.mark.gpu
E = 2.0 ** -24


def _dt(name):
    torch = H.torch_cuda()
    return torch.bfloat16 if name == "bf16" else torch.float32


def _round(a, dt):
    return H.torch_cuda().from_numpy(np.ascontiguousarray(a, np.float32)).to(dt).float().numpy()


def _case(rows, hs, dtype, dyt, seed, offset=0.25):
    g = np.random.default_rng(seed)
    x = _round(g.normal(size=(rows, hs)) * np.exp(0.5 * g.normal(size=hs)) + offset, _dt(dtype))
    dy = _round(g.normal(size=(rows, hs)), _dt(dyt))
    return x, dy, (1 + 0.3 * g.normal(size=hs)).astype(np.float32), g.normal(size=hs).astype(np.float32)


def run(x, dy, gamma, beta, dtype, dyt, eps=1e-5, pad=0, off=0, inplace="", sums=True, stream=None):
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    rows, hs = x.shape
    ld = hs + pad
    bf = dtype == "bf16"
    _, xv = _place(x, ld, off, _dt(dtype))
    ybuf, yv = _place(np.zeros((rows, hs), np.float32), ld + 3, off, _dt(dtype), fill=3.0)
    ga, be = (None if a is None else H.dev(a) for a in (gamma, beta))
    mu, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    torch.cuda.synchronize()
    f = vl.vl_layernorm_fwd_bf16 if bf else vl.vl_layernorm_fwd
    f(xv.data_ptr(), ld, rows, hs, ga, be, eps, yv.data_ptr(), ld + 3, mu, rstd, stream)
    out = {}
    if dy is not None:
        _, dyv = _place(dy, ld, off, _dt(dyt))
        dxbuf, dxv = _place(np.zeros((rows, hs), np.float32), ld + 3, off, _dt(dtype), fill=3.0)
        dxl = ld + 3
        if inplace:
            dxv, dxl = (xv if inplace == "x" else dyv), ld
        dg, db = torch.full((hs,), 9.0, device="cuda"), torch.full((hs,), 9.0, device="cuda")
        nb = vl.vl_layernorm_bwd_workspace_bytes(rows, hs)
        ws = torch.full((nb + 64,), 0xFF, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        a = (dyv.data_ptr(), ld, xv.data_ptr(), ld, rows, hs, ga, mu, rstd, dxv.data_ptr(), dxl)
        k = dict(dgamma=dg if sums else None, dbeta=db if sums else None, workspace=(ws.data_ptr(), nb), stream=stream)
        torch.cuda.synchronize()
        if bf:
            vl.vl_layernorm_bwd_bf16(*a, dy_f32=dyt == "f32", **k)
        else:
            vl.vl_layernorm_bwd(*a, **k)
        torch.cuda.synchronize()
        assert bool((ws[nb:] == 0xFF).all())
        if not inplace:
            assert bool((dxbuf[:off] == 3).all()) and bool((dxv[:, hs:] == 3).all())
        out = dict(dx=_wide(dxv, hs), dg=H.host(dg), db=H.host(db))
    torch.cuda.synchronize()
    assert bool((ybuf[:off] == 3).all()) and bool((yv[:, hs:] == 3).all())
    out.update(y=_wide(yv, hs), mu=H.host(mu), rstd=H.host(rstd))
    return out


def check(o, x, dy, gamma, beta, dtype, eps=1e-5, sums=True):
    rows, hs = x.shape
    ga = np.ones(hs) if gamma is None else gamma.astype(np.float64)
    be = np.zeros(hs) if beta is None else beta.astype(np.float64)
    y, mu, rstd = O.layernorm(x, ga, be, np.float32(eps))
    x = x.astype(np.float64)
    dmu = 128 * E * np.abs(x).mean(1) + 2 * E * np.abs(mu)
    _check(o["mu"], mu, dmu, "mu")
    drs = rstd * (136 * E + (dmu * rstd) ** 2)
    _check(o["rstd"], rstd, drs, "rstd")
    xh = (x - mu[:, None]) * rstd[:, None]
    tol = np.abs(ga) * (rstd * dmu)[:, None] + np.abs(xh * ga) * (144 * E) + 4 * E * (np.abs(be) + np.abs(y) + np.abs(ga * mu[:, None] * rstd[:, None]))
    check_rounded(o["y"], y, tol + E * np.abs(y), dtype, "y")
    if dy is not None:
        dy = dy.astype(np.float64)
        m32, r32 = o["mu"].astype(np.float64), o["rstd"].astype(np.float64)
        dx, dg, db = O.layernorm_bwd(dy, x, ga, m32, r32)
        xh = (x - m32[:, None]) * r32[:, None]
        exh = 4 * E * (np.abs(x) + np.abs(m32[:, None])) * r32[:, None]       # x - mu, rounded, times rstd
        t = dy * ga
        a, b = t.mean(1, keepdims=True), (t * xh).mean(1, keepdims=True)
        eb = 136 * E * np.abs(t * xh).mean(1, keepdims=True) + (np.abs(t) * exh).mean(1, keepdims=True)
        tol = r32[:, None] * (136 * E * np.abs(t).mean(1, keepdims=True) + np.abs(xh) * eb + np.abs(b) * exh +
                              8 * E * (np.abs(t) + np.abs(a) + np.abs(xh * b)))
        check_rounded(o["dx"], dx, tol + E * np.abs(dx), dtype, "dx")
        if sums:
            c = (rows / 32 + 64) * E
            _check(o["dg"], dg, c * np.abs(dy * xh).sum(0) + (np.abs(dy) * exh).sum(0), "dgamma")
            _check(o["db"], db, c * np.abs(dy).sum(0), "dbeta")


SIZES = [(1, 1), (3, 2), (1, 64), (5, 100), (37, 255), (9, 1000), (64, 768), (33, 1024), (200, 2050), (7, 4096), (5, 5003),
         (3, 8192), (4, 12288), (2, 16384), (3, 16383), (700, 513)]


@pytest.mark.parametrize("dtype,dyt", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("rows,hs", SIZES)
def test_norm(rows, hs, dtype, dyt):
    x, dy, ga, be = _case(rows, hs, dtype, dyt, rows + hs)
    o = run(x, dy, ga, be, dtype, dyt)
    check(o, x, dy, ga, be, dtype)


@pytest.mark.parametrize("dtype,dyt", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("rows,hs,pad,off", [(700, 64, 0, 0), (1300, 512, 0, 0), (640, 768, 8, 0), (640, 1024, 0, 8), (777, 2048, 0, 0),
                                             (615, 4096, 0, 0), (612, 5120, 16, 0), (611, 8192, 0, 0), (609, 8200, 0, 0),
                                             (609, 16384, 0, 0), (612, 2050, 0, 1), (613, 1500, 1, 0)])
def test_norm_of_many_rows(rows, hs, pad, off, dtype, dyt):
    """More rows than one CTA each takes at once: the persistent kernels, at every number of elements a thread."""
    x, dy, ga, be = _case(rows, hs, dtype, dyt, rows * hs)
    check(run(x, dy, ga, be, dtype, dyt, pad=pad, off=off), x, dy, ga, be, dtype)


@pytest.mark.parametrize("dtype,dyt", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("hs,pad,off", [(512, 0, 1), (512, 5, 0), (1000, 8, 8), (2051, 0, 3), (4096, 3, 2), (9001, 7, 1)])
def test_norm_strides_and_alignment(hs, pad, off, dtype, dyt):
    x, dy, ga, be = _case(11, hs, dtype, dyt, hs)
    check(run(x, dy, ga, be, dtype, dyt, pad=pad, off=off), x, dy, ga, be, dtype)
    check(run(x, dy, ga, be, dtype, dyt, pad=pad, off=off, inplace="x"), x, dy, ga, be, dtype)
    if dtype == dyt:
        check(run(x, dy, ga, be, dtype, dyt, pad=pad, off=off, inplace="dy"), x, dy, ga, be, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_without_affine_or_sums(dtype):
    x, dy, ga, be = _case(20, 1536, dtype, dtype, 2)
    check(run(x, dy, None, None, dtype, dtype), x, dy, None, None, dtype)
    o = run(x, dy, ga, None, dtype, dtype, sums=False)
    check(o, x, dy, ga, None, dtype, sums=False)
    assert (o["dg"] == 9).all() and (o["db"] == 9).all()


def test_norm_large_offset_flat_rows_and_specials():
    # a mean a thousand times the spread; a constant row (rstd = 1 / sqrt(eps)); NaN and inf stay in their rows
    x, dy, ga, be = _case(9, 3000, "f32", "f32", 4, offset=1000.0)
    x[3] = 2.5
    o = run(x, dy, ga, be, "f32", "f32")
    check(o, x, dy, ga, be, "f32")
    assert np.allclose(o["y"][3], be) and o["rstd"][3] == pytest.approx(1e-5 ** -0.5, rel=1e-6)
    x, dy, ga, be = _case(6, 3000, "f32", "f32", 4)
    x[1, 7], x[4, 2999] = np.nan, np.inf
    o = run(x, None, ga, be, "f32", "f32")
    keep = [0, 2, 3, 5]
    assert np.isnan(o["y"][1]).all() and np.isnan(o["y"][4]).all()
    check({k: v[keep] for k, v in o.items()}, x[keep], None, ga, be, "f32")


def test_norm_repeats_bit_for_bit_and_takes_other_streams():
    torch = H.torch_cuda()
    x, dy, ga, be = _case(5000, 1100, "bf16", "f32", 9)
    a = run(x, dy, ga, be, "bf16", "f32")
    b = run(x, dy, ga, be, "bf16", "f32", stream=torch.cuda.Stream())
    for k in a:
        assert np.array_equal(a[k], b[k]), k
    check(a, x, dy, ga, be, "bf16")


def test_norm_no_rows():
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    dg, db = torch.full((8,), 9.0, device="cuda"), torch.full((8,), 9.0, device="cuda")
    vl.vl_layernorm_bwd(None, 8, None, 8, 0, 8, None, None, None, None, 8, dg, db)
    torch.cuda.synchronize()
    assert not H.host(dg).any() and not H.host(db).any()


def test_norm_offsets_past_32_bits():
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    hs, ld = 512, (1 << 31) + 8
    buf = torch.zeros(2 * ld + hs, dtype=torch.bfloat16, device="cuda")
    g = np.random.default_rng(1)
    x = _round(g.normal(size=(3, hs)), torch.bfloat16)
    for t in range(3):
        buf[t * ld:t * ld + hs] = torch.from_numpy(x[t]).cuda().to(torch.bfloat16)
    mu, rstd = torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
    vl.vl_layernorm_fwd_bf16(buf, ld, 3, hs, None, None, 1e-5, buf, ld, mu, rstd)
    torch.cuda.synchronize()
    y = np.stack([buf[t * ld:t * ld + hs].float().cpu().numpy() for t in range(3)])
    check(dict(y=y, mu=H.host(mu), rstd=H.host(rstd)), x, None, None, None, "bf16")
