"""Bounded waits of kernels that start before their predecessor's end.

A kernel that calls pdl_wait_primary may be resident long before the work ahead of it is done.  Its producer issues no copy
before that, so a thread that already waits for the first one spends its limit on other kernels' time: were they to take
longer than the limit, the wait would run out and the kernel leave its outputs unwritten.  So every thread waits for the
work ahead first, in each of its roles.  Checked on the sources: a branch of a kernel that holds a bounded wait calls
pdl_wait_primary before it, if the kernel has not called it for all threads before.
"""
import os
import re

import pytest

from tests.test_wait_protocol import CSRC, _close, _functions, _plain

WAIT = re.compile(r"\bwait_(parity|all|one)\b")
START = "pdl_wait_primary"


def _blocks(body):
    """Spans of the braced blocks directly inside a function's body."""
    i = 1
    while (i := body.find("{", i)) >= 0:
        j = _close(body, i, "{}")
        yield i, j
        i = j


def early_waits(text):
    """Lines of bounded waits that come before the wait for the work ahead."""
    s = _plain(text)
    found = []
    for a, b in _functions(s):
        body = s[a:b]
        if START not in body:
            continue
        blocks = list(_blocks(body))
        inside = [False] * len(body)
        for p, q in blocks:
            inside[p:q] = [True] * (q - p)
        common = next((m.start() for m in re.finditer(START, body) if not inside[m.start()]), len(body))
        for p, q in blocks:
            wait = WAIT.search(body, p, q)
            if wait and p < common and not (0 <= body.find(START, p, q) < wait.start()):
                found.append(text[:a + wait.start()].count("\n") + 1)
    return found


def test_the_check_sees_such_a_wait():
    bad = """
    namespace vl {
    __global__ void f() {
        __syncthreads();
        if (warp == 0) {
            pdl_wait_primary();
            if (!wait_all(&S.empty[0], 0, &S.abort)) return;
        } else if (warp == 1) {
            for (int k = 0; k < 8; ++k)
                if (!wait_one(&S.full[k], 0, &S.abort)) break;   // pdl_wait_primary();
        }
    }
    }
    """
    assert early_waits(bad) == [10]
    assert early_waits(bad.replace("for (int k", "pdl_wait_primary(); for (int k")) == []
    assert early_waits(bad.replace("__syncthreads();", "pdl_wait_primary();")) == []
    assert early_waits(bad.replace("pdl_wait_primary();\n", "\n")) == []        # a kernel that does not start early
    assert early_waits(bad.replace("wait_one", "wait_parity_drain")) == []      # waits for copies issued, after all


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh"))))
def test_no_wait_before_the_work_ahead_is_done(name):
    with open(os.path.join(CSRC, name)) as f:
        assert early_waits(f.read()) == []
