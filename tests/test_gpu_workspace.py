"""The workspace that the binding keeps for a stream."""
import pytest

from tests import gpu_harness as H

pytestmark = pytest.mark.gpu


def _pairs(n, V, npairs):
    torch = H.torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randn(n, V, device="cuda", generator=g)
    lab = torch.randint(0, V, (n,), device="cuda", generator=g, dtype=torch.int32)
    start = (torch.arange(2 * npairs + 1, device="cuda", dtype=torch.int64) * n) // (2 * npairs)
    return x, lab, torch.ones(n, device="cuda"), start


def _preference(a, npairs, **k):
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    x, lab, w, start = a
    n, V = x.shape
    out = dict(grad=torch.empty_like(x), loss=torch.empty(npairs, device="cuda"), margin=torch.empty(npairs, device="cuda"),
               seq=torch.empty(2 * npairs, device="cuda"))
    torch.cuda.current_stream().synchronize()
    vl.vl_preference_loss(x, V, n, V, lab, w, start, npairs, None, 1e-3, 0.0, 0, 1.0, out["grad"], V, out["loss"],
                          out["margin"], out["seq"], **k)
    return out


def _norm(x, **k):
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    rows, hs = x.shape
    mu, rstd = x.mean(1), torch.rsqrt(x.var(1, correction=0) + 1e-5)
    out = dict(dx=torch.empty_like(x), dg=torch.empty(hs, device="cuda"), db=torch.empty(hs, device="cuda"))
    torch.cuda.current_stream().synchronize()
    vl.vl_layernorm_bwd(x, hs, x, hs, rows, hs, None, mu, rstd, out["dx"], hs, out["dg"], out["db"], **k)
    return out


@pytest.mark.parametrize("where", ["another", "default"])
@pytest.mark.parametrize("op", ["preference", "norm"])
def test_workspace_of_another_stream(op, where):
    """A call on another stream than torch's current one (the default one too) gets no memory that work queued on
    the current one still uses.

    A block of the workspace's size is freed while the kernels that write it are still queued; the
    allocator may give it to the stream it was freed on, and to no other."""
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    side = torch.cuda.Stream()
    current, s = (torch.cuda.default_stream(), side.cuda_stream) if where == "another" else (side, 0)
    if op == "preference":
        x, lab, w, start = _pairs(400000, 4, 50)
        need = vl.vl_preference_workspace_bytes(400000, 50)
        want = _preference((x, lab, w, start), 50, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
        outs = {k: torch.empty_like(v) for k, v in want.items()}

        def call():
            vl.vl_preference_loss(x, 4, 400000, 4, lab, w, start, 50, None, 1e-3, 0.0, 0, 1.0, outs["grad"], 4, outs["loss"],
                                  outs["margin"], outs["seq"], stream=s)
    else:
        x = torch.randn(20000, 4096, device="cuda")
        need = vl.vl_layernorm_bwd_workspace_bytes(20000, 4096)
        want = _norm(x, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
        outs = {k: torch.empty_like(v) for k, v in want.items()}
        mu, rstd = x.mean(1), torch.rsqrt(x.var(1, correction=0) + 1e-5)

        def call():
            vl.vl_layernorm_bwd(x, 4096, x, 4096, 20000, 4096, None, mu, rstd, outs["dx"], 4096, outs["dg"], outs["db"], stream=s)

    vl._stream_ws.pop((0, s), None)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(current):
        other = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
        busy = torch.empty(need, dtype=torch.uint8, device="cuda")
        at = busy.data_ptr()
        torch.cuda.synchronize()
        for _ in range(100):                                 # some milliseconds of writes
            other.fill_(1)
            busy.fill_(0xFF)
        del busy
        for _ in range(5):
            call()
    kept = vl._stream_ws[0, s]
    torch.cuda.synchronize()
    assert kept.data_ptr() >= at + need or at >= kept.data_ptr() + kept.numel()
    for k in want:
        assert torch.equal(outs[k], want[k]), k


def test_workspace_is_kept_and_grows():
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    s = torch.cuda.Stream()
    vl._stream_ws.pop((0, s.cuda_stream), None)
    small, large = _pairs(64, 8, 2), _pairs(4096, 8, 2)
    got = [_preference(a, 2, stream=st) for a in (small, large, small) for st in (s, s.cuda_stream)]
    torch.cuda.synchronize()
    assert len({k for k in vl._stream_ws if k[1] == s.cuda_stream}) == 1
    for a, o in zip((small, small, large, large, small, small), got):
        want = _preference(a, 2, workspace=torch.empty(vl.vl_preference_workspace_bytes(a[0].shape[0], 2), dtype=torch.uint8,
                                                       device="cuda"))
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(o[k], want[k]), k


def test_no_kept_workspace_in_a_captured_call():
    """A graph can be replayed on any stream, so it may not hold the buffer kept for one."""
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    a = _pairs(64, 8, 2)
    x, lab, w, start = a
    want = _preference(a, 2)
    out = [torch.empty_like(want[k]) for k in ("grad", "loss", "margin", "seq")]
    ws = torch.empty(vl.vl_preference_workspace_bytes(64, 2), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    before = set(vl._stream_ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(RuntimeError, match="workspace"):
            vl.vl_preference_loss(x, 8, 64, 8, lab, w, start, 2, None, 1e-3, 0.0, 0, 1.0, out[0], 8, *out[1:])
        with pytest.raises(RuntimeError, match="workspace"):
            vl.vl_layernorm_bwd(x, 8, x, 8, 64, 8, None, w, w, out[0], 8, out[1], out[1])
        vl.vl_preference_loss(x, 8, 64, 8, lab, w, start, 2, None, 1e-3, 0.0, 0, 1.0, out[0], 8, *out[1:], workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert before == set(vl._stream_ws)
    for k, t in zip(("grad", "loss", "margin", "seq"), out):
        assert torch.equal(t, want[k]), k


@pytest.mark.parametrize("where", ["another", "default"])
def test_topk_workspace_of_another_stream(where):
    """The cached buffer of the top-k calls: allocated on the call's stream, an outgrown one kept."""
    torch = H.torch_cuda()
    from top_kl_distill_gb300 import vloss as vl
    n, V, k = 300, 40000, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(n, V, device="cuda", generator=g)
    need = vl.vl_topk_workspace_bytes(n, V, k)
    want_p, want_i = torch.topk(x, k, dim=1)
    want_p = torch.softmax(want_p, 1)
    side = torch.cuda.Stream()
    current, s = (torch.cuda.default_stream(), side.cuda_stream) if where == "another" else (side, 0)
    held = vl._topk_ws.pop(0, None)                          # (kept alive: it may be in a graph)
    ids, probs = torch.empty(n, k, dtype=torch.int32, device="cuda"), torch.empty(n, k, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(current):
        other = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
        busy = torch.empty(need, dtype=torch.uint8, device="cuda")
        at = busy.data_ptr()
        torch.cuda.synchronize()
        for _ in range(100):
            other.fill_(1)
            busy.fill_(0)
        del busy
        vl.vl_topk_rows(x, V, n, V, k, 0, n, ids, probs, stream=s)
    first = vl.topk_workspace(1, 0)
    torch.cuda.synchronize()
    assert first.data_ptr() >= at + need or at >= first.data_ptr() + first.numel()
    assert torch.equal(ids.long(), want_i) and torch.allclose(probs, want_p, rtol=1e-5)
    grown = vl.topk_workspace(2 * first.numel(), 0)
    assert grown.data_ptr() != first.data_ptr() and vl.topk_workspace(1, 0) is grown
    assert any(t is first for t in vl._topk_ws[0])
    del held
