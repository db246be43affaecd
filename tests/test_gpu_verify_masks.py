"""Verification over rows whose masks are large finite numbers: the type's lowest value, -1e10, -1e30.

A masked column's weight is below 2^-149 of its row's, that is 0, exactly as for -inf, wherever the masked columns stand: the two
rows' results are the same bits.  Tokens are those of the float64 oracle for the rows masked with -inf.
"""
import numpy as np
import pytest

from tests import gpu_harness as H
from tests.test_gpu_verify import check, make, settle

pytestmark = pytest.mark.gpu

LOWEST = {"f32": float(np.finfo(np.float32).min), "bf16": -3.3895313892515355e38}


def call(t, y, s, tok, heat, u, pick, dtype):
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    n, nd, V = len(s) - 1, len(tok), t.shape[1]
    out = [torch.full((nd + n,), 77, dtype=torch.int32, device="cuda"), torch.full((n,), 77, dtype=torch.int32, device="cuda"),
           torch.full((nd + n,), 77.0, device="cuda")]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    (vl.vl_verify_draft_bf16 if dtype == "bf16" else vl.vl_verify_draft)(
        H.dev(t).to(dt), V, H.dev(y).to(dt) if y is not None else None, V, V, H.dev(s), n, nd, H.dev(tok),
        H.dev(heat) if heat is not None else None, H.dev(u), H.dev(pick), *out, err)
    torch.cuda.synchronize()
    return [H.host(o) for o in out] + [int(H.host(err)[0])]


@pytest.mark.parametrize("mask", ["lowest", -1e10, -1e30])
@pytest.mark.parametrize("temp", [None, [1.5, 2.0, 0.0], [0.7, 10.0, 30.0]])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masked_columns_weigh_nothing(mask, temp, draft, dtype):
    mask = LOWEST[dtype] if mask == "lowest" else mask
    for lens, V in (([4, 0, 3], 6000), ([2] * 60, 2500)):
        t, y, s, tok, h, u, p = make(lens, V, 21, temp=temp, draft=draft, dtype=dtype)
        away = np.zeros(V, bool)
        away[V // 8:V // 2] = True                               # whole segments and parts of them, the row's end
        away[-100:] = True
        away[np.random.default_rng(3).integers(0, V, V // 20)] = True
        away[tok] = False
        t[:, away] = -np.inf
        if draft:
            y[:, away] = -np.inf
        t, y, s, tok, h, u, p = settle(t, y, s, tok, h, u, p, np.random.default_rng(1))
        check(t, y, s, tok, h, u, p, dtype=dtype)
        want = call(t, y, s, tok, h, u, p, dtype)
        t = np.where(np.isinf(t), np.float32(mask), t)
        y = np.where(np.isinf(y), np.float32(mask), y) if draft else None
        got = call(t, y, s, tok, h, u, p, dtype)
        for a, b in zip(got, want):
            assert np.array_equal(a, b)


@pytest.mark.parametrize("temp", [1.0, 1.5, 30.0])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_column_left(temp, dtype):
    """Everything but one column at the type's lowest value, wherever that column stands."""
    V = 5000
    t = np.full((8, V), LOWEST[dtype], np.float32)
    at = np.array([0, 1, 1023, 1024, 2500, 4097, 4998, 4999])
    t[np.arange(8), at] = 1.0
    s = np.arange(5, dtype=np.int64)                             # one drafted token each: the column, and after it another row's
    tokens, acc, lp, err = call(t, None, s, at[::2].astype(np.uint32), np.full(4, temp, np.float32), np.full(4, 0.999, np.float32),
                                np.full(4, 0.5, np.float32), dtype)
    assert tokens.tolist() == at.tolist() and (acc == 1).all() and (lp == 0).all() and err == 0


@pytest.mark.parametrize("temp", [1.5, 2.0])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nothing_left(temp, dtype):
    """A row of nothing but the lowest value counts as masked throughout: it has no softmax, as a row of -inf."""
    t = np.full((2, 3000), LOWEST[dtype], np.float32)
    t[1, 7] = 0.0
    tokens, acc, lp, err = call(t, None, np.array([0, 0, 0], np.int64), np.zeros(0, np.uint32), np.full(2, temp, np.float32),
                                np.zeros(0, np.float32), np.full(2, 0.5, np.float32), dtype)
    assert tokens.view(np.uint32).tolist() == [0xFFFFFFFF, 7] and err == 1 and lp.tolist() == [0, 0]


@pytest.mark.parametrize("mask", ["lowest", -1e10, -1e30])
@pytest.mark.parametrize("temp", [1.0, 1.5, 0.3, 30.0, 0.0])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_drafted_tokens_that_are_masked(mask, temp, draft, dtype):
    """A token that the target bans is refused, whatever the drafter says of it and whatever u is; one that the drafter alone bans is
    accepted (p / 0): as with -inf."""
    mask = LOWEST[dtype] if mask == "lowest" else mask
    n, k, V = 24, 3, 3000
    t, y, s, tok, h, u, p = make([k] * n, V, 41, temp=[temp], draft=draft, dtype=dtype)
    rows = np.arange(n * k) + np.repeat(np.arange(n), k)
    for i in range(n * k):
        if i % 4 in (0, 1):                                      # the target's ban, and with it the drafter's or not
            t[rows[i], tok[i]] = -np.inf
        if draft and i % 4 in (1, 2):
            y[i, tok[i]] = -np.inf
    t[:, 2000:2300] = -np.inf
    if draft:
        y[:, 1990:2310] = -np.inf
    u[::5] = 0.0
    if temp != 0.0:
        t, y, s, tok, h, u, p = settle(t, y, s, tok, h, u, p, np.random.default_rng(1))
    want = call(t, y, s, tok, h, u, p, dtype)
    t = np.where(np.isinf(t), np.float32(mask), t)
    y = np.where(np.isinf(y), np.float32(mask), y) if draft else None
    got = call(t, y, s, tok, h, u, p, dtype)
    for i in range(n):                                           # none of the banned tokens comes out
        for j in range(int(got[1][i])):
            assert t[rows[k * i + j], tok[k * i + j]] > mask
    for a, b in zip(got, want):
        assert np.array_equal(a, b)
