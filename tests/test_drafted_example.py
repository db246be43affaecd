"""The example of drafted decoding: rows that do not fit its buffers are refused before anything is launched, and every token is
drawn by the library."""
import importlib.util
import os
import re
from types import SimpleNamespace

import pytest
import torch

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "drafted_decoding.py")


@pytest.fixture()
def ex(monkeypatch):
    spec = importlib.util.spec_from_file_location("drafted_decoding", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)

    def called(*a, **k):
        raise AssertionError("a launch")
    monkeypatch.setattr(m, "vl", SimpleNamespace(**{n: called for n in dir(m.vl) if n.startswith("vl_")}, VL_FP4_NV=0))
    return m


def rows(n, cols, dtype=torch.bfloat16):
    return torch.zeros(n, cols, dtype=dtype)


@pytest.fixture()
def step(ex):
    s = object.__new__(ex.Step)                       # without its buffers on the GPU
    s.head, s.y, s.out = SimpleNamespace(hs=8, V=10), rows(4, 8), rows(4, 10)
    return s


def test_rows_that_do_not_fit(ex, step):
    held = object.__new__(ex.Rows4)
    held.rows, held.cols = 4, 8
    for x in (rows(5, 8), rows(4, 7), rows(4, 16), rows(8, 4).t(), rows(4, 16)[:, :8], rows(1, 32)[0]):
        with pytest.raises(ValueError):
            held.take(x)
        with pytest.raises(ValueError):
            step.logits(x)


def test_counts_that_do_not_agree(step):
    i32 = torch.int32
    with pytest.raises(ValueError):                   # 4 hidden rows, but 3 drafted tokens and 2 sequences
        step.verify(rows(4, 8), None, torch.zeros(3, dtype=torch.int64), torch.zeros(3, dtype=i32), None, torch.zeros(3), torch.zeros(2),
                    torch.zeros(5, dtype=i32), torch.zeros(2, dtype=i32))
    for heat, pick, tokens in ((3, 4, 4), (4, 3, 4), (4, 4, 3)):
        with pytest.raises(ValueError):
            step.draw(rows(4, 8), torch.ones(heat), torch.zeros(pick), torch.zeros(tokens, dtype=i32))


def test_tokens_are_drawn_by_the_library():
    with open(PATH) as f:
        text = f.read()
    assert not re.search(r"softmax\(|multinomial\(|argmax\(|topk\(|matmul\(|layer_norm\(", text)
