"""Refusals of osdn_clip_grad_norm that depend on all of its tensors at once
(no GPU needed: nothing is dereferenced)."""
import ctypes
import math
import random

import pytest

from preconditioned_delta_rule_phase1_gb300 import build as osdn_build
from preconditioned_delta_rule_phase1_gb300 import ops

F = 0x100000
FINE = (-6, -10)   # no argument was refused: it got as far as the device check


@pytest.fixture(scope="module")
def L():
    osdn_build.build()
    return ops.lib()


def clip(L, g, o=None, sizes=None, ios=None, limit=1.0, norm=1 << 40, ws=1 << 41):
    n = len(g)
    sizes, ios = sizes or [16] * n, ios or [0] * n
    P = ctypes.c_void_p * n
    return L.osdn_clip_grad_norm(n, P(*g), None if o is None else P(*o), (ctypes.c_longlong * n)(*sizes),
                                 (ctypes.c_int * n)(*ios), limit, norm, ws, L.osdn_clip_grad_norm_workspace_bytes(n),
                                 None)


def test_outputs_that_are_other_gradients(L):
    a, b, c = F, 2 * F, 3 * F
    assert clip(L, [a, b], [b, a]) == -9                        # exchanged
    assert clip(L, [a, b, c], [b, 4 * F, 5 * F]) == -9
    assert clip(L, [a, b], [4 * F, a + 48]) == -9               # its last 16 bytes
    assert clip(L, [a, b], [4 * F, a + 64]) in FINE             # right behind it
    assert clip(L, [a, b], [4 * F, a + 48], sizes=[12, 16]) in FINE
    assert clip(L, [a, b], [4 * F, 4 * F + 32]) == -9           # two outputs
    assert clip(L, [a, b], [4 * F, 4 * F + 32], ios=[1, 0]) in FINE
    assert clip(L, [a, b], [a, b]) in FINE                      # in place
    assert clip(L, [a, a], [4 * F, 5 * F]) in FINE              # read twice
    assert clip(L, [a, b], [b, 4 * F], sizes=[0, 16]) in FINE   # nothing to write


def test_gradients_scaled_in_place(L):
    assert clip(L, [F, F]) == -9 and clip(L, [F, F + 32]) == -9 and clip(L, [F, F + 64]) in FINE
    assert clip(L, [F, F], limit=math.inf) in FINE and clip(L, [F, F + 32], limit=math.inf) in FINE
    assert clip(L, [F, F], [F, 2 * F], limit=math.inf) == -9    # the copy is written whatever the limit
    assert clip(L, [F], limit=math.inf, norm=F + 32) == -9 and clip(L, [F], limit=math.inf, ws=F + 32) == -9
    assert clip(L, [], norm=1 << 41) == -9                      # the norm inside the workspace
    assert clip(L, [F, 0], sizes=[16, 0]) in FINE


def test_elements_of_all_tensors(L):
    # chunks of 8192 elements are numbered in 32 bits over a launch's tensors
    big, at = 1 << 40, [(i + 1) << 44 for i in range(40)]
    assert clip(L, at[:16], sizes=[big] * 16, norm=F, ws=2 * F) in FINE
    assert clip(L, at[:17], sizes=[big] * 16 + [1], norm=F, ws=2 * F) == -2
    assert clip(L, at[:33], sizes=[big] * 33, norm=F, ws=2 * F) == -2


def test_against_pairs(L):
    # more tensors than are sorted at once, in any order; overlaps of a few bytes
    rng = random.Random(1)
    for n, outs in ((3, True), (40, True), (40, False), (700, True), (1600, False), (2500, True)):
        for hits in (0, 0, 1, 1, 2):
            m = n * (2 if outs else 1)
            sizes = [rng.choice([0, 1, 4, 16, 100]) for _ in range(n)]
            at, p = F, [0] * m
            for k in rng.sample(range(m), m):
                p[k] = at
                at += -(-sizes[k % n] * 4 // 16) * 16 + rng.choice([0, 0, 64])
            for _ in range(hits):
                i, j = rng.sample(range(m), 2)
                p[i] = p[j] + rng.choice([0, 16])
            span = [(p[k], p[k] + 4 * sizes[k % n], not outs or k >= n) for k in range(m)]
            # an output on its own gradient is the call in place
            span = [(lo, hi, w or (outs and p[k] == p[k + n])) if k < n else (lo, lo if p[k] == p[k - n] else hi, w)
                    for k, (lo, hi, w) in enumerate(span)]
            span = sorted(s for s in span if s[0] < s[1])
            # sorted by start, so two overlap only if a later one starts before an earlier one's end
            hit = any(a[1] > b[0] and (a[2] or b[2]) for i, a in enumerate(span) for b in span[i + 1:i + 30])
            got = clip(L, p[:n], p[n:] if outs else None, sizes)
            assert got == -9 if hit else got in FINE, (n, outs, hits)
