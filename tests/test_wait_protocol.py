"""A wait that ran out must not part threads that meet at a barrier.

Every wait of the kernels is bounded; one that gives up says so, and what goes by its answer may leave
a loop.  Threads of other warps may have seen the same wait succeed: if the loop holds a barrier of
several warps, they would wait there for ever for those that left.  So no loop that holds such a
barrier may end by the answer of a wait.  Checked on the sources: loops that hold a barrier, by their
condition and by the conditions of their own break and return statements.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "top_kl_distill_gb300", "csrc")
BARRIER = re.compile(r"\b(named_sync\w*|__syncthreads\w*|cluster_sync_all)\s*\(")
WAIT = re.compile(r"\bwait_(parity|all)\b")


def _plain(text):
    """The source without comments, strings and preprocessor lines, of the same length."""
    def blank(m):
        return re.sub(r"[^\n]", " ", m.group(0))
    text = re.sub(r"//[^\n]*|/\*.*?\*/", blank, text, flags=re.S)
    text = re.sub(r'"(\\.|[^"\\\n])*"', blank, text)
    return re.sub(r"(?m)^[ \t]*#(.*\\\n)*.*$", blank, text)


def _close(s, i, pair="()"):
    """The index past the bracket that closes the one at i."""
    depth = 0
    for j in range(i, len(s)):
        depth += (s[j] == pair[0]) - (s[j] == pair[1])
        if depth == 0:
            return j + 1
    raise AssertionError("unbalanced source")


def _statement(s, i):
    """The index past the statement that begins at i."""
    while s[i].isspace():
        i += 1
    if s[i] == "{":
        return _close(s, i, "{}")
    m = re.compile(r"(if\s*(constexpr)?|for|while|switch)\s*\(").match(s, i)
    if m:
        j = _statement(s, _close(s, m.end() - 1))
        e = re.compile(r"\s*else\b").match(s, j)
        return _statement(s, e.end()) if m.group(1).startswith("if") and e else j
    j = i
    while s[j] != ";":
        j = _close(s, j, "{}") if s[j] == "{" else _close(s, j) if s[j] == "(" else j + 1
    return j + 1


def _loops(s):
    """(start, header, body span) of every for and while loop."""
    for m in re.finditer(r"\b(for|while)\s*\(", s):
        h = _close(s, m.end() - 1)
        yield m.start(), s[m.end():h - 1], (h, _statement(s, h))


def _functions(s):
    """Spans of the outermost bodies inside namespaces: functions (and types, which hold no loops)."""
    i = 0
    while (i := s.find("{", i)) >= 0:
        if re.search(r"(namespace[\w\s]*|extern\s*)$", s[:i]):
            i += 1
            continue
        j = _close(s, i, "{}")
        yield i, j
        i = j


def _answers(body):
    """Names that hold, or may be set by, the answer of a wait in this function."""
    names = set(re.findall(r"\b(\w+)\s*=\s*[^;=]*\bwait_(?:parity|all)\b", body))
    names = {n[0] if isinstance(n, tuple) else n for n in names}
    for m in re.finditer(r"\bif\s*\(", body):                # if (!wait...) { flag = ...; }
        c = _close(body, m.end() - 1)
        if WAIT.search(body[m.end():c]):
            names |= set(re.findall(r"\b(\w+)\s*=(?!=)", body[c:_statement(body, c)]))
    for m in re.finditer(r"\b(\w+)\s*=\s*__all_sync\s*\([^,]*,\s*(\w+)\s*\)", body):
        if m.group(2) in names:
            names.add(m.group(1))
    return names


def parting_loops(text):
    """Lines of loops that hold a barrier and end by the answer of a wait."""
    s = _plain(text)
    found = []
    for a, b in _functions(s):
        body = s[a:b]
        names = _answers(body)
        asks = re.compile(WAIT.pattern + "".join(r"|\b%s\b" % n for n in sorted(names)))
        for at, header, (p, q) in _loops(body):
            inside = body[p:q]
            if not BARRIER.search(inside):
                continue
            condition = header.split(";")[1] if header.count(";") == 2 else header
            ends = bool(asks.search(condition))
            nested = [span for _, _, span in _loops(inside)]
            for m in re.finditer(r"\bif\s*\(", inside):
                c = _close(inside, m.end() - 1)
                then = inside[c:_statement(inside, c)]
                own = not any(x <= m.start() < y for x, y in nested)
                leaves = re.search(r"\breturn\b", then) or own and re.search(r"\bbreak\b", then)
                ends = ends or bool(leaves and asks.search(inside[m.end():c]))
            if ends:
                found.append(text[:a + at].count("\n") + 1)
    return found


def test_the_check_sees_such_a_loop():
    bad = """
    namespace vl {
    __device__ void f(uint64_t* bar) {
        bool stop = false;
        for (int t = 0; t < n && !stop; ++t) {
            named_sync(1, 128);                 // a comment: break
            for (int k = 0; k < 8; ++k) {
                if (!wait_all(bar, k & 1)) {
                    stop = true;
                    break;
                }
            }
        }
    }
    }
    """
    assert parting_loops(bad) == [5]
    assert parting_loops(bad.replace(" && !stop", "")) == []
    assert parting_loops(bad.replace("&& !stop; ++t) {", "; ++t) { if (stop) break;")) == [5]
    assert parting_loops(bad.replace("named_sync(1, 128)", "__syncwarp()")) == []
    assert parting_loops("void g() { bool ok = wait_parity(b); while (ok) { __syncthreads(); } }") == [1]


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh"))))
def test_no_wait_parts_threads_that_meet(name):
    with open(os.path.join(CSRC, name)) as f:
        assert parting_loops(f.read()) == []
