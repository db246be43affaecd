"""One post-training step at the vocabulary head, through the library's calls alone:

    hidden rows -> layer norm -> 8-bit product with the frozen head -> policy or preference loss,
    its gradient written over the logits -> 8-bit product back -> layer norm's backward pass

``Head`` holds the frozen plane in 8 bits, both ways round, and ``Step`` the buffers of a batch,
so that a step allocates nothing and can be captured in a CUDA graph.  Run as a program it
trains a small model's hidden rows and norm on synthetic tokens, first against a reward, then on
pairs, and prints how both come along:

    python examples/post_training.py [--rows 256 --hidden 512 --vocab 512 --steps 40]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from top_kl_distill_gb300 import vloss as vl  # noqa: E402


def _blocks(n):
    return -(-n // 128)


class Head:
    """A frozen head plane w [V][hs] (bf16; hs a multiple of 16), quantised once: as it is for the logits, and
    transposed for the way back, with columns of zeros up to ld, the next multiple of 16 from V."""

    def __init__(self, w):
        self.V, self.hs = w.shape
        self.ld = -(-self.V // 16) * 16
        self.plane = self._quantise(w)
        self.back = self._quantise(torch.nn.functional.pad(w.t(), (0, self.ld - self.V)).contiguous())

    @staticmethod
    def _quantise(w):
        n, k = w.shape
        q = torch.empty(n, k, dtype=torch.uint8, device=w.device)
        s = torch.empty(_blocks(n), _blocks(k), device=w.device)
        vl.vl_quant_fp8_blocks_bf16(w, n, k, q, s)
        return q, s


class Step:
    """The buffers of a step over n rows, and the step itself."""

    def __init__(self, head, n):
        ld, hs = head.ld, head.hs
        self.head, self.n = head, n

        def f32(*shape):
            return torch.empty(*shape, device="cuda")

        def u8(*shape):
            return torch.empty(*shape, dtype=torch.uint8, device="cuda")

        self.y = torch.empty(n, hs, dtype=torch.bfloat16, device="cuda")
        self.mu, self.rstd = f32(n), f32(n)
        self.yq, self.ys = u8(n, hs), f32(_blocks(hs), n)
        # the gradient, after the loss; the columns of padding stay zero (nothing writes them)
        self.logits = torch.zeros(n, ld, device="cuda")[:, :head.V]
        self.gq, self.gs = u8(n, ld), f32(_blocks(ld), n)
        self.dy = f32(n, hs)
        self.dx = torch.empty(n, hs, dtype=torch.bfloat16, device="cuda")
        self.dgamma, self.dbeta = f32(hs), f32(hs)
        self.loss, self.logp, self.kl = f32(n), f32(n), f32(n)
        self.total = f32(1)
        self.norm_ws = u8(max(16, vl.vl_layernorm_bwd_workspace_bytes(n, hs)))
        self.pair_ws = u8(max(16, vl.vl_preference_workspace_bytes(n, max(1, n // 2))))

    def logits_of(self, x, gamma, beta, eps=1e-5):
        """The logits of hidden rows x [n][hs] bf16."""
        h, n = self.head, self.n
        vl.vl_layernorm_fwd_bf16(x, h.hs, n, h.hs, gamma, beta, eps, self.y, h.hs, self.mu, self.rstd)
        vl.vl_quant_fp8_rows_bf16(self.y, h.hs, n, h.hs, self.yq, self.ys)
        vl.vl_gemm_fp8_tn(self.yq, self.ys, *h.plane, self.logits, n, h.V, h.hs, h.ld)
        return self.logits

    def backward(self, x, gamma):
        """From the gradient that a loss left in the logits' place: dx, dgamma, dbeta."""
        h, n = self.head, self.n
        vl.vl_quant_fp8_rows(self.logits, h.ld, n, h.ld, self.gq, self.gs)
        vl.vl_gemm_fp8_tn(self.gq, self.gs, *h.back, self.dy, n, h.hs, h.ld, h.hs)
        vl.vl_layernorm_bwd_bf16(self.dy, h.hs, x, h.hs, n, h.hs, gamma, self.mu, self.rstd, self.dx, h.hs, self.dgamma,
                                 self.dbeta, workspace=self.norm_ws)
        return self.dx, self.dgamma, self.dbeta

    def policy(self, x, gamma, beta, actions, old_logp, ref_logp, adv, weight, clip=(0.2, 0.2), kl_coef=0.04):
        """A policy step: total [1] and per-row loss, logp, kl stay in the buffers; returns the gradients."""
        s, V, ld = self.logits_of(x, gamma, beta), self.head.V, self.head.ld
        vl.vl_policy_loss(s, ld, self.n, V, actions, old_logp, ref_logp, adv, weight, *clip, kl_coef, 1.0, s, ld,
                          self.loss, self.logp, self.kl, self.total)
        return self.backward(x, gamma)

    def preference(self, x, gamma, beta, labels, weight, seq_start, npairs, ref_logp, loss, margin, seq_logp,
                   strength=0.1, kind=0):
        """A preference step over npairs pairs (kind: 0 sigmoid, 1 squared, 2 hinge); returns the gradients."""
        s, V, ld = self.logits_of(x, gamma, beta), self.head.V, self.head.ld
        vl.vl_preference_loss(s, ld, self.n, V, labels, weight, seq_start, npairs, ref_logp, strength, 0.0, kind,
                              1.0 / npairs, s, ld, loss, margin, seq_logp, self.total, workspace=self.pair_ws)
        return self.backward(x, gamma)


def _descend(lr, params, grads):
    """Plain signed descent on master copies (what optimiser a model uses is its own affair)."""
    for p, g in zip(params, grads):
        p.sub_(lr * g.float().sign())


def train_policy(rows, hs, V, steps, lr=0.02, seed=1):
    """Mean probability of the rewarded tokens, before and after.  Tokens with an even number are rewarded."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    head = Head((torch.randn(V, hs, device="cuda", generator=g) * hs ** -0.5).to(torch.bfloat16))
    step = Step(head, rows)
    x = torch.randn(rows, hs, device="cuda", generator=g)
    gamma, beta = torch.ones(hs, device="cuda"), torch.zeros(hs, device="cuda")
    weight = torch.full((rows,), 1.0 / rows, device="cuda")

    def rewarded():
        p = torch.softmax(step.logits_of(x.to(torch.bfloat16), gamma, beta), 1)
        return float(p[:, ::2].sum(1).mean())

    before, ref = rewarded(), None
    for _ in range(steps):
        xb = x.to(torch.bfloat16)
        logp = torch.log_softmax(step.logits_of(xb, gamma, beta), 1)
        act = torch.multinomial(logp.exp(), 1, generator=g)
        old = logp.gather(1, act)[:, 0].contiguous()
        ref = logp.clone() if ref is None else ref          # the first policy is the reference
        adv = torch.where(act[:, 0] % 2 == 0, 1.0, -1.0)
        grads = step.policy(xb, gamma, beta, act[:, 0].to(torch.int32), old,
                            ref.gather(1, act)[:, 0].contiguous(), adv, weight)
        _descend(lr, (x, gamma, beta), grads)
    return before, rewarded()


def train_preference(pairs, length, hs, V, steps, lr=0.02, seed=2):
    """(mean loss, mean margin) before the first and the last update."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    head = Head((torch.randn(V, hs, device="cuda", generator=g) * hs ** -0.5).to(torch.bfloat16))
    n = 2 * pairs * length
    step = Step(head, n)
    x = torch.randn(n, hs, device="cuda", generator=g)
    gamma, beta = torch.ones(hs, device="cuda"), torch.zeros(hs, device="cuda")
    labels = torch.randint(0, V, (n,), device="cuda", generator=g, dtype=torch.int32)
    weight = (torch.arange(n, device="cuda") % length >= length // 4).float()      # the first quarter is the prompt
    start = torch.arange(2 * pairs + 1, device="cuda", dtype=torch.int64) * length
    logp = torch.log_softmax(step.logits_of(x.to(torch.bfloat16), gamma, beta), 1)
    ref = (logp.gather(1, labels.long()[:, None])[:, 0] * weight).view(2 * pairs, length).sum(1).contiguous()
    loss, margin, pi = (torch.empty(k, device="cuda") for k in (pairs, pairs, 2 * pairs))
    seen = []
    for _ in range(steps):
        grads = step.preference(x.to(torch.bfloat16), gamma, beta, labels, weight, start, pairs, ref, loss, margin, pi)
        seen.append((float(step.total), float(margin.mean())))
        _descend(lr, (x, gamma, beta), grads)
    return seen[0], seen[-1]


def main():
    a = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    a.add_argument("--rows", type=int, default=256)
    a.add_argument("--hidden", type=int, default=512)
    a.add_argument("--vocab", type=int, default=512)
    a.add_argument("--steps", type=int, default=40)
    o = a.parse_args()
    was, now = train_policy(o.rows, o.hidden, o.vocab, o.steps)
    print(f"policy: probability of rewarded tokens {was:.3f} -> {now:.3f}")
    first, last = train_preference(max(1, o.rows // 32), 16, o.hidden, o.vocab, o.steps)
    print(f"preference: loss {first[0]:.4f} -> {last[0]:.4f}, margin {first[1]:.3f} -> {last[1]:.3f}")


if __name__ == "__main__":
    main()
