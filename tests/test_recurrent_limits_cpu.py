"""The sizes and workspaces that the recurrent layer's calls take and refuse (no GPU needed:
a call that is not refused stops at the device check, before anything is enqueued)."""
import types

import pytest
import torch

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


BIG = (1 << 32) + 16   # cut down to 32 bits: 16


def test_sizes_that_do_not_fit_the_c_calls_are_refused_by_the_binding(L):
    """Not passed on as what is left of them in 32 bits."""
    new = lambda *shape, dtype=torch.float32: torch.empty(*shape, dtype=dtype, device="meta")  # noqa: E731
    calls = []
    for shape in ((1, BIG, 1), (BIG, 1, 1), (1, 1, BIG)):
        x = new(*shape)
        calls += [lambda x=x: ops.gated_scan(x, x), lambda x=x: ops.gated_scan_backward(x, x, x, dh=x)]
    for shape in ((BIG, 1), (1, BIG)):
        x = new(*shape)
        calls += [lambda x=x: ops.gated_scan_step(x, x, x)]
    x = new(1, BIG)
    calls += [lambda: ops.layer_norm(x), lambda: ops.layer_norm_backward(x, x)]
    for call in calls:
        with pytest.raises(ops.OsdnError) as e:
            call()
        assert e.value.code == -2


def test_a_workspace_of_another_device_is_refused(L):
    """By the calls that need none, too, as by those that do."""
    x = torch.zeros(2, 5, 64)
    elsewhere = types.SimpleNamespace(buf=torch.empty(256, dtype=torch.uint8, device="meta"))
    here = types.SimpleNamespace(buf=torch.empty(256, dtype=torch.uint8))
    for call in (lambda ws: ops.gated_scan(x, x, workspace=ws),
                 lambda ws: ops.gated_scan_backward(x, x, x, dh=x, workspace=ws),
                 lambda ws: ops.layer_norm_backward(x, x, workspace=ws)):
        with pytest.raises(ValueError, match="workspace is on meta"):
            call(elsewhere)
        with pytest.raises(ValueError, match="CUDA tensors only"):   # no argument was refused
            call(here)
