"""The example of drafted decoding draws every token by the library."""
import os
import re

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "drafted_decoding.py")


def test_tokens_are_drawn_by_the_library():
    with open(PATH) as f:
        text = f.read()
    assert not re.search(r"softmax\(|multinomial\(|argmax\(|topk\(|matmul\(|layer_norm\(", text)
