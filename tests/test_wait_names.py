"""Waits go by names that the check of the wait protocol knows.

That check follows the answers of wait_parity and wait_all.  A helper of another name that hands such an answer on would hide it:
functions that return one are called wait_parity or wait_all themselves.
"""
import os
import re

import pytest

from tests.test_wait_protocol import CSRC, WAIT, _functions, _plain


def hidden_waits(text):
    """Names of functions that return a wait's answer and are not called as the check expects."""
    s = _plain(text)
    found = []
    for a, b in _functions(s):
        head = re.search(r"\bbool\s+(\w+)\s*\([^{};]*\)\s*$", s[:a])
        if head and re.search(r"\breturn\b[^;]*" + WAIT.pattern, s[a:b]) and not WAIT.fullmatch(head.group(1)):
            found.append(head.group(1))
    return found


def test_the_check_sees_such_a_function():
    text = "namespace vl {\n__device__ bool %s(uint64_t* b, int* a) {\n    return __all_sync(~0u, wait_parity<false>(b, 0, a, &flag));\n}\n}"
    assert hidden_waits(text % "wait_one") == ["wait_one"]
    assert hidden_waits(text % "wait_all") == []
    assert hidden_waits((text % "wait_one").replace("wait_parity", "wait_parity_drain")) == []


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh"))))
def test_waits_are_known_by_their_names(name):
    with open(os.path.join(CSRC, name)) as f:
        assert hidden_waits(f.read()) == []
