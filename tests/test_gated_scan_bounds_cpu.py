"""Accesses of the gated recurrence that no result shows (no GPU needed: the
sources are read).

A lane owns channels c and c + 1.  In rows of an odd number of channels the last
lane's second one does not exist: reading it is reading the next sequence's
first channel, or past the end of the tensor behind the last sequence.  The value
is used for nothing, so no comparison can see it, and a GPU shows it only where
the tensor ends with a mapping, by a fault.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "preconditioned_delta_rule_phase1_gb300", "csrc")


def source(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


@pytest.mark.parametrize("name", ["gated_scan.cu", "gated_scan_backward.cu"])
def test_states_are_read_and_written_channel_by_channel_that_exists(name):
    """The [B][C] fp32 tensors (h0, dhT; hT, dh0) go through load_state and store_state alone."""
    uses = re.findall(r"[^\n]*\bp\.(?:first|h0|last)\b[^\n]*", source(name))
    kernel = [u for u in uses if not re.search(r"p\.(first|h0|last) = ", u)]   # (the host fills them in)
    assert kernel
    for u in kernel:
        assert re.search(r"load_state\(p, p\.(first|h0)\)|store_state\(p, p\.last, s\)", u), u


def test_load_and_store_look_at_both_channels():
    text = source("gated_scan_walk.cuh")
    for name, first, second in (("load_state", r"if \(s && live\) v\.v\[0\] = s\[", r"if \(s && second\) v\.v\[1\] = s\["),
                                ("store_state", r"if \(s && live\) s\[", r"if \(s && second\) s\[")):
        body = text[text.index(name + "("):]
        body = body[:body.index("\n    }")]
        assert re.search(first, body) and re.search(second, body), name
        assert len(re.findall(r"\bs\[", body)) == 2, name
    assert re.search(r"live = c < p\.C;", text) and re.search(r"second = c \+ 1 < p\.C;", text)
