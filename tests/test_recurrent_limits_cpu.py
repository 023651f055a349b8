"""The sizes that the gated recurrence's C entry points take and refuse (no GPU needed:
a call that is not refused stops at the device check, before anything is enqueued)."""
import pytest

from preconditioned_delta_rule_phase1_gb300 import build as osdn_build
from preconditioned_delta_rule_phase1_gb300 import ops

F = 1 << 44          # addresses a terabyte and more apart, never dereferenced
FINE = (-6, -10)     # no argument was refused: it got as far as the device check
MANY = 2147483647


@pytest.fixture(scope="module")
def L():
    osdn_build.build()
    return ops.lib()


def scan(L, B, T, C):
    return L.osdn_gated_scan(1, B, T, C, 1, F, 2 * F, 3 * F, 4 * F, 5 * F, None)


def back(L, B, T, C):
    return L.osdn_gated_scan_backward(1, B, T, C, 1, *[i * F for i in range(1, 10)], None)


def test_many_short_and_narrow_sequences_are_taken(L):
    """The number of sequences alone does not bound a call: 2^30 of 17 tokens of a channel are 37 GB."""
    for call in (scan, back):
        for B, T, C in ((1 << 30, 17, 1), (MANY, 1, 1), (MANY, 15, 1), (1 << 26, 33, 33), (1, 1073741760, 256),
                        (1 << 17, 1, 1 << 19)):
            assert call(L, B, T, C) in FINE, (call, B, T, C)
    assert L.osdn_gated_scan_step(1, MANY, 64, 1, F, 2 * F, 3 * F, 4 * F, None) in FINE


def test_what_cannot_be_numbered_is_refused(L):
    for call in (scan, back):
        for B, T, C in ((MANY, 1, 65), (1 << 25, 1, 1 << 13), (1, 1073741761, 1), (1, 1, (1 << 24) + 1),
                        (1 << 20, 1 << 20, 1), (1, 1073741760, 1024)):
            assert call(L, B, T, C) == -2, (call, B, T, C)
