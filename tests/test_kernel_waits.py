"""How the delta kernels' roles end when a wait runs out, read from their sources (no GPU needed;
a wait that runs out is not staged on one).

Warps that work as a whole (tensor-memory loads and stores are instructions of all 32 lanes) and
groups that meet at a named barrier must not lose a lane or a warp on the way: each thread's wait runs
out by its own clock, and whoever stayed would wait for the one that left without a limit.  So their
loops have a fixed number of turns, and nothing leaves them early.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), os.pardir,
                    "weight_state_recurrence_b200", "csrc")
FILES = ["delta_tc.cuh", "delta_bwd_tc.cuh"]
COLLECTIVE = re.compile(r"\b(tmem_ld\w*|tmem_st\w*|named_bar_sync|__syncthreads|__shfl\w*)\b")
LEAVES = re.compile(r"\b(break|return|goto)\b")


def closing(s, i):
    """Index behind the bracket that closes the one at i."""
    pairs = {"(": ")", "{": "}", "[": "]"}
    stack = []
    for j in range(i, len(s)):
        if s[j] in pairs:
            stack.append(pairs[s[j]])
        elif stack and s[j] == stack[-1]:
            stack.pop()
            if not stack:
                return j + 1
    raise AssertionError("unbalanced")


def loops(s):
    """(header, body) of every for loop with a body in braces, comments taken out."""
    s = re.sub(r"//[^\n]*", "", s)
    for m in re.finditer(r"\bfor \(", s):
        end = closing(s, m.end() - 1)
        rest = re.match(r"\s*\{", s[end:])
        if rest:
            at = end + rest.end() - 1
            yield s[m.end():end - 1], s[at:closing(s, at)]


def test_the_loops_are_found():
    body = "for (int i = 0; ok && i < n; ++i) { if (x) break; tmem_ld<16>(a, d); } // for (a) {"
    assert list(loops(body)) == [("int i = 0; ok && i < n; ++i", "{ if (x) break; tmem_ld<16>(a, d); }")]


@pytest.mark.parametrize("name", FILES)
def test_no_lane_leaves_a_loop_of_whole_warps(name):
    with open(os.path.join(CSRC, name)) as f:
        found = [(h, b) for h, b in loops(f.read()) if COLLECTIVE.search(b)]
    assert len(found) > 4
    for header, body in found:
        assert "ok" not in header, f"a wait's outcome ends the loop: for ({header})"
        assert not LEAVES.search(body), f"left early: for ({header})"


def kernel(name, text):
    """The body of the kernel `name`."""
    at = text.index("{", closing(text, text.index("(", text.index(f" {name}("))))
    return text[at:closing(text, at)]


@pytest.mark.parametrize("name,source,bars", [("delta_prep_kernel", "delta_tc.cuh", ["bar_load"]),
                                              ("delta_grad_kernel", "delta_bwd_tc.cuh",
                                               ["b_in", "b_s", "b_d"])])
def test_copies_under_way_are_waited_for_again(name, source, bars):
    # a copy that lands after its block has gone would write into the next one's shared memory
    with open(os.path.join(CSRC, source)) as f:
        body = kernel(name, re.sub(r"//[^\n]*", "", f.read()))
    end = body.rindex("if (!ok)")
    for bar in bars:
        assert len(re.findall(rf"\b(?:tma_load_3d|bulk_load|load_state)\([^;]*\b{bar}\b", body)) > 0
        assert f"mbar_wait({bar}, 0)" in body[end:]
