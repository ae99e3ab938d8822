"""What the MXFP4 grouped kernel does with the results of its bounded waits, read from its source.

A wait that runs out ends the kernel with a status.  Nothing that a caller passes makes one run
out, so the rules of that path are checked where they are written."""
import os
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "routing_grouped_gemm_gb300",
                   "csrc", "grouped_mx.cu")
VOTE = re.compile(r"__all_sync|__shfl_sync|__any_sync")
WARP_WIDE = re.compile(r"\b(bar_and|bar_sync|elect_one|cluster_sync|tc_fence_after|tmem_ld\w*|tmem_dealloc\w*|__syncthreads)\s*\(")


def _waits():
    """(start of the statement, start of the call, end of the call) of every wait."""
    text = re.sub(r"//[^\n]*", lambda m: " " * len(m.group()), open(SRC).read())
    out = []
    for m in re.finditer(r"\bmbar_wait_bounded\s*\(", text):
        depth, i = 0, m.end() - 1
        while True:
            depth += {"(": 1, ")": -1}.get(text[i], 0)
            i += 1
            if depth == 0:
                break
        start = max(text.rfind(c, 0, m.start()) for c in ";{}") + 1
        out.append((start, m.start(), i))
    return text, out


def test_lanes_agree_on_a_wait_before_anything_warp_wide():
    """The wait's loop has several exits for each lane; the .aligned forms want the warp together."""
    text, waits = _waits()
    assert len(waits) >= 7
    for start, call, end in waits:
        line = text.count("\n", 0, call) + 1
        if VOTE.search(text, start, call):
            continue
        vote, wide = VOTE.search(text, end), WARP_WIDE.search(text, end)
        assert vote and (not wide or vote.start() < wide.start()), f"line {line}"


def test_no_wait_is_left_without_a_look_at_its_result():
    """Tensor memory that is freed after a wait that ran out is reported."""
    text, waits = _waits()
    for start, call, _ in waits:
        assert text[start:call].strip(), f"line {text.count(chr(10), 0, call) + 1}"


@pytest.mark.parametrize("name", ["grouped_mx", "grouped_tc", "grouped_tc2", "grouped_bwd", "router"])
def test_a_drain_that_runs_out_is_reported(name):
    """The wait for the MMAs in flight before a CTA frees tensor memory, in every tcgen05 kernel."""
    text = open(os.path.join(os.path.dirname(SRC), name + ".cu")).read()
    waits = re.findall(r"^.*(?:wait_drained\(|mbar_wait_bounded\((?:drain|done), 0u, &local_abort).*$", text, re.M)
    assert waits
    for w in waits:
        assert "wait_drained(" in w or w.strip().startswith("if (!") and w.strip().endswith("*abort_flag = 1;"), w
