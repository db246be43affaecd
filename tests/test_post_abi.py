"""The post-training entry points refuse bad arguments on the host, before anything is launched."""
import pytest

from top_kl_distill_gb300 import vloss as vl

P = 1 << 20          # never dereferenced
FAR = 1 << 40


def _status(fn, *a, **k):
    with pytest.raises(vl.VlossError) as e:
        fn(*a, **k)
    assert fn.__name__ in str(e.value)
    return e.value.status


def _policy(fn=vl.vl_policy_loss, logits=P, ld=10, ntok=4, V=10, act=P, old=P, ref=None, adv=P, w=P, lo=0.2, hi=0.2, kl=0.0,
            grad=FAR, ldg=10, loss=P):
    return fn, logits, ld, ntok, V, act, old, ref, adv, w, lo, hi, kl, 1.0, grad, ldg, loss, None, None, None, None, 0


@pytest.mark.parametrize("bad", [dict(ld=9), dict(V=0), dict(ntok=-1), dict(logits=None), dict(act=None), dict(old=None),
                                 dict(adv=None), dict(w=None), dict(loss=None), dict(lo=-0.1), dict(lo=1.5), dict(hi=-1.0),
                                 dict(lo=float("nan")), dict(hi=float("nan")), dict(ldg=9), dict(grad=P + 4),
                                 dict(grad=P, ldg=12), dict(grad=P - 4), dict(V=vl.VL_MAX_COLS + 1, ld=1 << 31)])
@pytest.mark.parametrize("fn", [vl.vl_policy_loss, vl.vl_policy_loss_bf16])
def test_policy_refuses(fn, bad):
    assert _status(*_policy(fn, **bad)) == vl.VL_EINVAL


def test_policy_takes_nothing():
    f, *a = _policy(ntok=0, logits=None, act=None, old=None, adv=None, w=None, loss=None, grad=None, ldg=0)
    f(*a)


def _pref(fn=vl.vl_preference_loss, logits=P, ld=10, ntok=4, V=10, lab=P, w=P, start=P, pairs=1, ref=None, beta=0.1,
          smooth=0.0, kind=0, grad=FAR, ldg=10, loss=P, margin=P, ws=(P, 1 << 20)):
    return (fn, logits, ld, ntok, V, lab, w, start, pairs, ref, beta, smooth, kind, 1.0, grad, ldg, loss, margin, None, None,
            None, ws, 0)


@pytest.mark.parametrize("bad", [dict(ld=9), dict(V=0), dict(logits=None), dict(lab=None), dict(w=None), dict(start=None),
                                 dict(loss=None), dict(margin=None), dict(pairs=-1), dict(pairs=0), dict(beta=0.0),
                                 dict(beta=float("nan")), dict(beta=float("inf")), dict(smooth=1.0), dict(smooth=-0.1),
                                 dict(kind=3), dict(kind=-1), dict(ldg=9), dict(grad=P + 8), dict(ws=None),
                                 dict(ws=(P, 63)), dict(ws=(P + 8, 1 << 20))])
@pytest.mark.parametrize("fn", [vl.vl_preference_loss, vl.vl_preference_loss_bf16])
def test_preference_refuses(fn, bad):
    assert _status(*_pref(fn, **bad)) == vl.VL_EINVAL


def test_preference_workspace():
    f = vl.vl_preference_workspace_bytes
    assert f(0, 0) == 0 and f(-3, 1) == 0 and 0 < f(1, 1) <= f(1000, 3) <= f(1000, 300) and f(4, 1) >= 64


def _fwd(x=P, ldx=8, rows=4, hs=8, eps=1e-5, y=FAR, ldy=8):
    return x, ldx, rows, hs, None, None, eps, y, ldy, None, None, 0


@pytest.mark.parametrize("bad", [dict(x=None), dict(y=None), dict(ldx=7), dict(ldy=7), dict(rows=-1), dict(hs=0),
                                 dict(eps=-1.0), dict(eps=float("nan")), dict(y=P + 4), dict(y=P, ldy=9)])
@pytest.mark.parametrize("fn", [vl.vl_layernorm_fwd, vl.vl_layernorm_fwd_bf16])
def test_norm_forward_refuses(fn, bad):
    assert _status(fn, *_fwd(**bad)) == vl.VL_EINVAL


def test_norm_limits():
    big = vl.VL_NORM_MAX_HS + 1
    assert _status(vl.vl_layernorm_fwd, *_fwd(hs=big, ldx=big, ldy=big)) == vl.VL_EUNSUPPORTED
    assert vl.vl_layernorm_bwd_workspace_bytes(5, big) == 0 == vl.vl_layernorm_bwd_workspace_bytes(0, 8)
    vl.vl_layernorm_fwd(*_fwd(rows=0, x=None, y=None))


def _bwd(dy=FAR, lddy=8, x=P, ldx=8, rows=4, hs=8, mu=P, rstd=P, dx=2 * FAR, lddx=8, dg=P, db=P, ws=(P, 1 << 20)):
    return dy, lddy, x, ldx, rows, hs, None, mu, rstd, dx, lddx, dg, db, ws, 0


@pytest.mark.parametrize("bad", [dict(dy=None), dict(x=None), dict(dx=None), dict(mu=None), dict(rstd=None), dict(lddy=7),
                                 dict(ldx=7), dict(lddx=7), dict(dx=P + 4), dict(dx=FAR, lddx=9), dict(ws=None),
                                 dict(ws=(P, 8)), dict(ws=(P + 8, 1 << 20))])
def test_norm_backward_refuses(bad):
    assert _status(vl.vl_layernorm_bwd, *_bwd(**bad)) == vl.VL_EINVAL
    if bad != dict(dx=FAR, lddx=9):
        assert _status(vl.vl_layernorm_bwd_bf16, *_bwd(**bad), dy_f32=False) == vl.VL_EINVAL
    with pytest.raises(ValueError):
        vl.vl_layernorm_bwd_bf16(*_bwd())
    # a bf16 dx may not stand where the fp32 dy is
    assert _status(vl.vl_layernorm_bwd_bf16, *_bwd(dx=FAR), dy_f32=True) == vl.VL_EINVAL


def test_quantisers_refuse():
    for fn in (vl.vl_quant_fp8_rows, vl.vl_quant_fp8_rows_bf16):
        assert _status(fn, None, 16, 4, 16, P, P, 0) == vl.VL_EINVAL
        assert _status(fn, P, 15, 4, 16, P, P, 0) == vl.VL_EINVAL
        assert _status(fn, P, 16, -1, 16, P, P, 0) == vl.VL_EINVAL
        assert _status(fn, P, 16, 4, 16, P, None, 0) == vl.VL_EINVAL
        fn(None, 16, 0, 16, None, None, 0)
    assert _status(vl.vl_quant_fp8_blocks_bf16, P, 4, 16, None, P, 0) == vl.VL_EINVAL
    vl.vl_quant_fp8_blocks_bf16(None, 0, 16, None, None, 0)


@pytest.mark.parametrize("bad", [dict(K=24), dict(K=0), dict(M=-1), dict(ldd=7), dict(A=None), dict(sa=None), dict(sb=None),
                                 dict(B=P + 8), dict(D=None)])
def test_product_refuses(bad):
    a = dict(A=P, sa=P, B=P, sb=P, D=P, M=4, N=8, K=32, ldd=8)
    a.update(bad)
    assert _status(vl.vl_gemm_fp8_tn, *a.values(), 1.0, 0) == vl.VL_EINVAL


def test_empty_product_launches_nothing():
    vl.vl_gemm_fp8_tn(P, P, P, P, P, 0, 8, 32, 8, 1.0, 0)
    vl.vl_gemm_fp8_tn(P, P, P, P, P, 4, 0, 32, 8, 1.0, 0)
