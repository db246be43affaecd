"""Drafted decoding at the vocabulary head, through the library's calls alone: a small student proposes tokens, its teacher
looks at all of them in one pass and keeps what it would have said itself:

    hidden rows -> layer norm -> 4-bit rows -> 4-bit product with the student's head
           -> a token each (verification of nothing drafted), token by token
    hidden rows of all drafted positions -> layer norm -> 4-bit rows -> 4-bit product with the teacher's head
           -> verification against the student's logits, from given random numbers

``Head`` holds a head plane in 4 bits, ``Step`` the buffers of a pass, so that a pass allocates nothing and can be captured
in a CUDA graph.  Run as a program it decodes with a random teacher (a token's next hidden row hangs on the token alone) and
a student that is the teacher with some noise, and prints how many tokens a pass of the teacher gives:

    python examples/drafted_decoding.py [--seqs 16 --drafted 4 --hidden 512 --vocab 2000 --passes 20 --noise 0.3 --heat 0.8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from top_kl_distill_gb300 import vloss as vl  # noqa: E402


class Rows4:
    """Buffers of [rows][cols] in 4 bits: values, scales of blocks of 16, scales of rows."""

    def __init__(self, rows, cols):
        self.rows, self.cols = rows, cols
        self.q = torch.empty(rows, -(-cols // 32) * 16, dtype=torch.uint8, device="cuda")
        self.sf = torch.empty(vl.vl_fp4_scale_bytes(rows, cols, vl.VL_FP4_NV), dtype=torch.uint8, device="cuda")
        self.rs = torch.empty(rows, device="cuda")

    def take(self, x):
        """Quantises bf16 rows x [n <= rows][cols]."""
        if x.dim() != 2 or x.shape[0] > self.rows or x.shape[1] != self.cols or not x.is_contiguous():
            raise ValueError(f"rows {tuple(x.shape)} do not fit buffers of [{self.rows}][{self.cols}]")
        vl.vl_quant_fp4_rows_bf16(x, self.cols, x.shape[0], self.cols, vl.VL_FP4_NV, self.q, self.sf, self.rs)
        return self


class Head:
    """A head plane w [V][hs] (bf16), quantised once, with the layer norm before it."""

    def __init__(self, w, gamma, beta):
        self.V, self.hs = w.shape
        self.gamma, self.beta = gamma, beta
        self.plane = Rows4(self.V, self.hs).take(w)


class Step:
    """The buffers of a pass over up to `rows` hidden rows, and the pass itself."""

    def __init__(self, head, rows):
        self.head = head
        self.y = torch.empty(rows, head.hs, dtype=torch.bfloat16, device="cuda")
        self.x4 = Rows4(rows, head.hs)
        self.out = torch.empty(rows, head.V, dtype=torch.bfloat16, device="cuda")
        self.none = torch.zeros(rows + 1, dtype=torch.int64, device="cuda")           # starts of sequences with nothing drafted
        self.nil = torch.empty(rows, dtype=torch.int32, device="cuda")

    def logits(self, x):
        """Logits (bf16) of hidden rows x [n][hs] bf16."""
        h, n = self.head, x.shape[0]
        if x.dim() != 2 or n > self.y.shape[0] or x.shape[1] != h.hs or not x.is_contiguous():
            raise ValueError(f"hidden rows {tuple(x.shape)} do not fit a step of [{self.y.shape[0]}][{h.hs}]")
        y, out = self.y[:n], self.out[:n]
        vl.vl_layernorm_fwd_bf16(x, h.hs, n, h.hs, h.gamma, h.beta, 1e-5, y, h.hs)
        self.x4.take(y)
        vl.vl_gemm_fp4_tn_bf16(self.x4.q, self.x4.sf, self.x4.rs, h.plane.q, h.plane.sf, h.plane.rs, out, n, h.V, h.hs, h.V,
                               vl.VL_FP4_NV)
        return out

    def draw(self, x, heat, pick, tokens):
        """A token for each hidden row, from its softmax at temperature heat[i] and the random number pick[i]."""
        n, V = x.shape[0], self.head.V
        if not n == heat.numel() == pick.numel() == tokens.numel():
            raise ValueError(f"{n} hidden rows, {heat.numel()} temperatures, {pick.numel()} random numbers, {tokens.numel()} tokens")
        t = self.logits(x)
        vl.vl_verify_draft_bf16(t, V, None, V, V, self.none, n, 0, None, heat, None, pick, tokens, self.nil)
        return t

    def verify(self, x, draft, start, drafted, heat, u, pick, tokens, accepted, logp=None):
        """One pass of the teacher: hidden rows x of the drafted positions and of the one after them, sequence by
        sequence; the drafter's logits (None: proposals without probabilities), its tokens and the random numbers."""
        if x.shape[0] != drafted.numel() + pick.numel():
            raise ValueError(f"{x.shape[0]} hidden rows for {drafted.numel()} drafted tokens of {pick.numel()} sequences")
        t, V = self.logits(x), self.head.V
        vl.vl_verify_draft_bf16(t, V, draft, V, V, start, pick.numel(), drafted.numel(), drafted, heat, u, pick, tokens, accepted, logp)
        return t


def decode(seqs, k, hs, V, passes, noise, heat, seed=1):
    """(tokens a pass and sequence, share of drafted tokens accepted, the sequences' last tokens)."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*s):
        return torch.randn(*s, device="cuda", generator=g)

    table = rand(V, hs).to(torch.bfloat16)                          # a token's hidden row
    w = (2 * hs ** -0.5 * rand(V, hs)).to(torch.bfloat16)
    gamma, beta = torch.ones(hs, device="cuda"), torch.zeros(hs, device="cuda")
    teacher = Step(Head(w, gamma, beta), seqs * (k + 1))
    student = Step(Head((w + noise * 2 * hs ** -0.5 * rand(V, hs)).to(torch.bfloat16), gamma, beta), seqs)
    start = torch.arange(seqs + 1, device="cuda", dtype=torch.int64) * k
    temp = torch.full((seqs,), heat, device="cuda")
    draft = torch.empty(seqs, k, V, dtype=torch.bfloat16, device="cuda")
    drafted = torch.empty(seqs, k, dtype=torch.int32, device="cuda")
    tokens = torch.empty(seqs, k + 1, dtype=torch.int32, device="cuda")
    accepted = torch.empty(seqs, dtype=torch.int32, device="cuda")
    said = torch.empty(seqs, dtype=torch.int32, device="cuda")
    last, kept, given = torch.randint(0, V, (seqs,), device="cuda", generator=g), 0, 0
    for _ in range(passes):
        seen = torch.empty(seqs, k + 1, dtype=torch.int64, device="cuda")
        seen[:, 0] = last
        for j in range(k):                                          # the student goes ahead, token by token
            draft[:, j] = student.draw(table[seen[:, j]], temp, torch.rand(seqs, device="cuda", generator=g), said)
            seen[:, j + 1] = said
        drafted.copy_(seen[:, 1:])
        u, pick = (torch.rand(n, device="cuda", generator=g) for n in (seqs * k, seqs))
        teacher.verify(table[seen.view(-1)], draft.view(seqs * k, V), start, drafted.view(-1), temp, u, pick, tokens.view(-1), accepted)
        last = tokens.gather(1, accepted.long()[:, None])[:, 0].long()
        kept += int(accepted.sum())
        given += int(accepted.sum()) + seqs
    return given / passes / seqs, kept / (passes * seqs * k), last


def main():
    a = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    a.add_argument("--seqs", type=int, default=16)
    a.add_argument("--drafted", type=int, default=4)
    a.add_argument("--hidden", type=int, default=512)
    a.add_argument("--vocab", type=int, default=2000)
    a.add_argument("--passes", type=int, default=20)
    a.add_argument("--noise", type=float, default=0.3)
    a.add_argument("--heat", type=float, default=0.8)
    o = a.parse_args()
    each, share, _ = decode(o.seqs, o.drafted, o.hidden, o.vocab, o.passes, o.noise, o.heat)
    print(f"{each:.2f} tokens a pass and sequence; {100 * share:.0f}% of the drafted tokens accepted")


if __name__ == "__main__":
    main()
