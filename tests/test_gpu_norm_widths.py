"""Layer norm at every access width and number of elements a thread, over enough rows that each group
goes round its ring of rows in flight, against float64 on the GPU.

x, dy, y and dx get the same stride, so that 16-byte accesses are taken wherever hs allows them: at a
stride of its own for y (as test_gpu_norm.py places it) the forward pass goes by single elements.
Tolerances as there: sums off by 136 * 2^-24 of their terms' sizes, column sums by
(rows / 32 + 64) * 2^-24 of theirs, a few 2^-24 of the terms elementwise; bf16 outputs between the
bf16 roundings of the fp32 interval's ends.
"""
import pytest

from tests import gpu_harness as H
from tests.post_plain import _near, _near_rounded

pytestmark = pytest.mark.gpu
E = 2.0 ** -24


def _view(rows, hs, ld, off, dt):
    torch = H.torch_cuda()
    buf = torch.full((off + rows * ld + 16,), 3.0, dtype=dt, device="cuda")
    return buf, buf[off:off + rows * ld].view(rows, ld)[:, :hs]


def check(rows, hs, dtype, dyt, pad=0, off=0, back=True, inplace=False, eps=1e-5):
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    g = torch.Generator(device="cuda").manual_seed(rows * 7 + hs)
    dt, ddt = (torch.bfloat16 if t == "bf16" else torch.float32 for t in (dtype, dyt))
    bf, ld = dtype == "bf16", hs + pad

    def rand(*s):
        return torch.randn(*s, device="cuda", generator=g)

    _, xv = _view(rows, hs, ld, off, dt)
    xv.copy_(rand(rows, hs) * torch.exp(0.5 * rand(hs)) + 0.25)
    x = xv.double()
    ga, be = 1 + 0.3 * rand(hs), rand(hs)
    ybuf, yv = _view(rows, hs, ld, off, dt)
    mu, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    f = vl.vl_layernorm_fwd_bf16 if bf else vl.vl_layernorm_fwd
    f(xv.data_ptr(), ld, rows, hs, ga, be, eps, yv.data_ptr(), ld, mu, rstd)
    torch.cuda.synchronize()
    g64, b64 = ga.double(), be.double()
    var, m64 = torch.var_mean(x, 1, correction=0)
    r64 = (var + float(torch.tensor(eps))).rsqrt()
    dmu = 128 * E * x.abs().mean(1) + 2 * E * m64.abs()
    _near(mu, m64, dmu, "mu")
    _near(rstd, r64, r64 * (136 * E + (dmu * r64) ** 2), "rstd")
    xh = (x - m64[:, None]) * r64[:, None]
    y = xh * g64 + b64
    tol = (g64.abs() * (r64 * dmu)[:, None] + (xh * g64).abs() * (144 * E) +
           4 * E * (b64.abs() + y.abs() + (g64 * m64[:, None] * r64[:, None]).abs()) + E * y.abs())
    _near_rounded(yv, y, tol, "y")
    assert bool((ybuf[:off] == 3).all()) and bool((ybuf[off + rows * ld:] == 3).all())
    if pad:
        assert bool((ybuf[off:off + rows * ld].view(rows, ld)[:, hs:] == 3).all())
    if not back:
        return
    _, dyv = _view(rows, hs, ld, off, ddt)
    dyv.copy_(rand(rows, hs))
    dy = dyv.double()
    dxv = xv if inplace else _view(rows, hs, ld, off, dt)[1]
    dg, db = torch.full((hs,), 9.0, device="cuda"), torch.full((hs,), 9.0, device="cuda")
    nb = vl.vl_layernorm_bwd_workspace_bytes(rows, hs)
    ws = torch.full((nb + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    a = (dyv.data_ptr(), ld, xv.data_ptr(), ld, rows, hs, ga, mu, rstd, dxv.data_ptr(), ld, dg, db)
    torch.cuda.synchronize()
    if bf:
        vl.vl_layernorm_bwd_bf16(*a, workspace=(ws.data_ptr(), nb), dy_f32=dyt == "f32")
    else:
        vl.vl_layernorm_bwd(*a, workspace=(ws.data_ptr(), nb))
    torch.cuda.synchronize()
    assert bool((ws[nb:] == 0xFF).all())
    m32, r32 = mu.double()[:, None], rstd.double()[:, None]
    xh = (x - m32) * r32
    exh = 4 * E * (x.abs() + m32.abs()) * r32
    t = dy * g64
    p, q = t.mean(1, keepdim=True), (t * xh).mean(1, keepdim=True)
    dx = r32 * (t - p - xh * q)
    eq = 136 * E * (t * xh).abs().mean(1, keepdim=True) + (t.abs() * exh).mean(1, keepdim=True)
    tol = r32 * (136 * E * t.abs().mean(1, keepdim=True) + xh.abs() * eq + q.abs() * exh +
                 8 * E * (t.abs() + p.abs() + (xh * q).abs())) + E * dx.abs()
    _near_rounded(dxv, dx, tol, "dx")
    c = (rows / 32 + 64) * E
    _near(dg, (dy * xh).sum(0), c * (dy * xh).abs().sum(0) + (dy.abs() * exh).sum(0), "dgamma")
    _near(db, dy.sum(0), c * dy.abs().sum(0), "dbeta")


TYPES = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")]


# 16, 24, 32 and (bf16, 16-byte rows) 64 elements a thread; the rows are more than every group of the device holds
# in its ring at once, so that stages are used again and again
@pytest.mark.parametrize("dtype,dyt", TYPES)
@pytest.mark.parametrize("rows,hs", [(40000, 64), (30000, 512), (20000, 768), (20000, 1024), (16000, 2048), (12000, 2304),
                                     (9000, 4096), (4000, 8192), (3000, 12288), (2500, 16384)])
def test_wide_rows_round_the_ring(rows, hs, dtype, dyt):
    check(rows, hs, dtype, dyt)


# two elements at a time, and one
@pytest.mark.parametrize("dtype,dyt", TYPES)
@pytest.mark.parametrize("rows,hs,pad,off", [(9000, 2050, 0, 0), (20000, 514, 0, 2), (3000, 10002, 0, 0), (9000, 2051, 0, 0),
                                             (20000, 333, 0, 1), (2500, 16383, 1, 0), (6000, 4096, 2, 0), (6000, 4096, 8, 8)])
def test_narrow_accesses_round_the_ring(rows, hs, pad, off, dtype, dyt):
    check(rows, hs, dtype, dyt, pad=pad, off=off)


# a row a CTA: one, two and four vectors a thread, one row and the most
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 8, 608])
@pytest.mark.parametrize("hs", [8, 1000, 2048, 4096, 8192, 16384])
def test_few_rows(rows, hs, dtype):
    check(rows, hs, dtype, dtype)


@pytest.mark.parametrize("dtype,dyt", TYPES)
@pytest.mark.parametrize("rows,hs", [(9000, 4096), (9000, 2050), (2500, 16384)])
def test_many_rows_in_place(rows, hs, dtype, dyt):
    check(rows, hs, dtype, dyt, inplace=True)
