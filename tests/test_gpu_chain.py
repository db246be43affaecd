"""Chains of calls over one set of buffers whose contents change from step to step: every call reads what
the one before it in the stream wrote, in an eager loop and in a graph.

A kernel of the chain starts while its predecessor still runs, so what it reads has to be read after
that one's end, past any cache that an earlier step filled.
"""
import pytest

from tests import gpu_harness as H

pytestmark = pytest.mark.gpu


class Chain:
    """scale gamma -> layer norm -> row quantiser -> product -> (its quantiser) -> layer norm backward."""

    def __init__(self, rows, hs, V):
        torch = H.torch_cuda()
        self.rows, self.hs, self.V = rows, hs, V
        g = torch.Generator(device="cuda").manual_seed(rows + V)

        def rand(*s):
            return torch.randn(*s, device="cuda", generator=g)

        self.gammas, self.betas = 1 + 0.5 * rand(STEPS, hs), rand(STEPS, hs)
        self.inputs = (rand(STEPS, rows, hs) * torch.exp(rand(STEPS, 1, 1))).to(torch.bfloat16)
        self.planes = rand(STEPS, V, hs).to(torch.bfloat16)
        self.gamma, self.beta = torch.empty(hs, device="cuda"), torch.empty(hs, device="cuda")
        self.x, self.w = torch.empty_like(self.inputs[0]), torch.empty_like(self.planes[0])
        self.y, self.dx = torch.empty_like(self.x), torch.empty_like(self.x)
        self.mu, self.rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")

        def plane(n, k):
            return torch.empty(n, k, dtype=torch.uint8, device="cuda")

        kb, vb = -(-hs // 128), -(-V // 128)
        self.q, self.s = plane(rows, hs), torch.empty(kb, rows, device="cuda")
        self.wq, self.ws = plane(V, hs), torch.empty(vb, kb, device="cuda")
        self.d = torch.empty(rows, V, device="cuda")
        self.dq, self.ds = plane(rows, V), torch.empty(vb, rows, device="cuda")
        self.dgamma, self.dbeta = torch.empty(hs, device="cuda"), torch.empty(hs, device="cuda")
        from top_kl_distill_gb300 import vloss as vl
        self.vl = vl
        self.wsp = torch.empty(max(16, vl.vl_layernorm_bwd_workspace_bytes(rows, hs)), dtype=torch.uint8, device="cuda")

    def load(self, i):
        self.gamma.copy_(self.gammas[i])
        self.beta.copy_(self.betas[i])
        self.x.copy_(self.inputs[i])
        self.w.copy_(self.planes[i])

    def calls(self):
        vl, r, h, v = self.vl, self.rows, self.hs, self.V
        return [
            lambda: vl.vl_quant_fp8_blocks_bf16(self.w, v, h, self.wq, self.ws),
            lambda: vl.vl_layernorm_fwd_bf16(self.x, h, r, h, self.gamma, self.beta, 1e-5, self.y, h, self.mu, self.rstd),
            lambda: vl.vl_quant_fp8_rows_bf16(self.y, h, r, h, self.q, self.s),
            lambda: vl.vl_gemm_fp8_tn(self.q, self.s, self.wq, self.ws, self.d, r, v, h, v),
            lambda: vl.vl_quant_fp8_rows(self.d, v, r, v, self.dq, self.ds),
            lambda: vl.vl_layernorm_bwd_bf16(self.y, h, self.x, h, r, h, self.gamma, self.mu, self.rstd, self.dx, h, self.dgamma,
                                             self.dbeta, workspace=self.wsp),
            # the affine's own update, and the next step's first half straight after it
            lambda: vl.vl_acc_add(self.gamma, self.dgamma, h),
            lambda: vl.vl_layernorm_fwd_bf16(self.x, h, r, h, self.gamma, self.dbeta, 1e-5, self.y, h, self.mu, self.rstd),
            lambda: vl.vl_quant_fp8_rows_bf16(self.y, h, r, h, self.q, self.s),
            lambda: vl.vl_gemm_fp8_tn(self.q, self.s, self.wq, self.ws, self.d, r, v, h, v),
        ]

    def outputs(self):
        return [t.clone() for t in (self.y, self.mu, self.q, self.s, self.wq, self.ws, self.d, self.dq, self.ds, self.dx,
                                    self.dgamma, self.dbeta)]


STEPS = 6


# the products: few rows (two CTAs an SM), pairs of CTAs; norms: a row a CTA, the persistent kernels with
# gamma in registers and (16384) from memory
@pytest.mark.parametrize("rows,hs,V", [(8, 512, 1040), (8, 4096, 4000), (60, 1024, 20000), (200, 768, 1500), (700, 256, 2064),
                                       (160, 16384, 272)])
def test_chained_steps(rows, hs, V):
    torch = H.torch_cuda()
    c = Chain(rows, hs, V)
    want = []
    for i in range(STEPS):                                   # each call waited for
        c.load(i)
        for f in c.calls():
            torch.cuda.synchronize()
            f()
        torch.cuda.synchronize()
        want.append(c.outputs())
    got = []
    for i in range(STEPS):
        c.load(i)
        for f in c.calls():
            f()
        got.append(c.outputs())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for f in c.calls():
            f()
    replayed = []
    for i in range(STEPS):
        c.load(i)
        graph.replay()
        replayed.append(c.outputs())
    torch.cuda.synchronize()
    for i in range(STEPS):
        for k, (a, b, d) in enumerate(zip(want[i], got[i], replayed[i])):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), ("eager", i, k)
            assert torch.equal(a.view(torch.uint8), d.view(torch.uint8)), ("graph", i, k)
    assert not torch.equal(want[0][6], want[1][6])


def test_captured_steps_follow_one_another():
    """Several steps in one graph, each with inputs of its own copied in between."""
    torch = H.torch_cuda()
    c = Chain(8, 4096, 8000)
    outs = [torch.empty_like(c.d) for _ in range(STEPS)]
    want = []
    for i in range(STEPS):
        c.load(i)
        for f in c.calls():
            torch.cuda.synchronize()
            f()
        want.append(c.d.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(STEPS):
            c.load(i)
            for f in c.calls():
                f()
            outs[i].copy_(c.d)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, outs):
        assert torch.equal(a, b)
