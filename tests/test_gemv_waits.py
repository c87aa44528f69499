"""The few-row kernels' bounded waits, read from the source (no GPU: a wait
that runs out cannot be provoked through the library's calls, and the failure
would be a hang). A wait ends for each thread by itself, by the phase or by the
abort flag; code of whole warps goes on to barriers, so there the warp has to
vote. Every plain wait must therefore stand in code of one thread."""
from __future__ import annotations

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gemm_pt_block_gb300", "csrc")


def blocks_around(text, at):
    """The headers (text before the brace) of the blocks around a position, and
    the condition of its own statement."""
    stack = []
    start = 0
    for i in range(at):
        c = text[i]
        if c == "{":
            stack.append(text[start:i])
        elif c == "}":
            stack.pop()
        if c in "{};":
            start = i + 1
    return stack + [text[start:at]]


def source():
    with open(os.path.join(CSRC, "gemv.cu")) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def waits(text):
    return [m.start() for m in re.finditer(r"\bwait_bar\s*(<\w+>)?\s*\(", text)]


def test_plain_waits_stand_in_code_of_one_thread():
    text = source()
    found = 0
    for at in waits(text):
        around = blocks_around(text, at)
        if re.search(r"bool\s+$", text[max(0, at - 40):at]) or any("wait_bar_warp" in b for b in around):
            continue                                       # the definitions
        found += 1
        one = any("lane == 0" in b for b in around) or any("void produce(" in b for b in around)
        assert one, text[text.rfind("\n", 0, at):text.find("\n", at)]
    assert found >= 5


def test_the_one_thread_functions_are_called_by_one_thread():
    text = source()
    calls = [m.start() for m in re.finditer(r"\bproduce\s*<", text)]
    assert len(calls) == 2
    for at in calls:
        assert any("lane == 0" in b for b in blocks_around(text, at))


@pytest.mark.parametrize("snippet,ok", [
    ("void k() { if (lane == 0) { wait_bar(a, b, c); } }", True),
    ("void k() { for (;;) { if (!wait_bar(a, b, c)) break; } }", False),
])
def test_the_reading_itself(snippet, ok):
    at = waits(snippet)[0]
    assert any("lane == 0" in b for b in blocks_around(snippet, at)) == ok
