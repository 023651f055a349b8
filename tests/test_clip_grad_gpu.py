"""Global gradient norm and clipping (osdn_clip_grad_norm) against 64-bit sums.

Tolerances: the norm is summed with its rounding errors kept and rounded to
fp32 once, 2e-7; the scale is rounded to fp32 and each product to its type.
"""
import math

import pytest
import torch

from preconditioned_delta_rule_phase1_gb300 import build as osdn_build
from preconditioned_delta_rule_phase1_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    osdn_build.build()
    ops.lib()


def norm64(gs):
    return math.sqrt(math.fsum(float(g.double().square().sum()) for g in gs))


def tensors(sizes, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * scale).to(torch.bfloat16 if i % 3 else torch.float32)
            for i, n in enumerate(sizes)]


SIZES = [[1], [7], [8191], [8192], [8193], [16384, 1, 0, 50000], [3, 5, 7] * 30, [1000003, 17, 262144],
         [100 + i for i in range(2100)]]   # the last: three tables


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "%d tensors of %d" % (len(s), s[0]))
def test_norm_and_clipping(sizes):
    gs = tensors(sizes)
    n = norm64(gs)
    assert abs(float(ops.grad_norm(gs)) - n) < 2e-7 * n
    ws = ops.Workspace()
    for limit in (0.25 * n, 4.0 * n):
        c = min(1.0, limit / n)
        outs = [torch.full_like(g, 5.0) for g in gs]
        before = [g.clone() for g in gs]
        got = ops.clip_grad_norm(gs, limit, outs=outs, workspace=ws)
        assert abs(float(got) - n) < 2e-7 * n
        assert all(torch.equal(g, b) for g, b in zip(gs, before))
        inplace = [g.clone() for g in gs]
        ops.clip_grad_norm(inplace, limit, workspace=ws)
        for g, o, p in zip(gs, outs, inplace):
            assert torch.equal(o, p)
            if not g.numel():
                continue
            if c == 1.0:
                assert torch.equal(o, g)
            else:
                ulp = 2.0 ** -8 if g.dtype == torch.bfloat16 else 2.0 ** -22
                assert ((o.double() - g.double() * c).abs() <= ulp * (g.double() * c).abs()).all()


def test_values_outside_the_range_of_squares():
    # squares over 3e38 and under 1e-45: the norm itself is an fp32 number
    for scale in (1e25, 1e-25, 1e18, 1e-20):
        gs = tensors([5000, 20000, 3], seed=1, scale=scale)
        n = norm64(gs)
        assert abs(float(ops.grad_norm(gs)) - n) < 2e-7 * n, scale
        outs = [torch.empty_like(g) for g in gs]
        ops.clip_grad_norm(gs, 1.0, outs=outs)
        assert abs(norm64(outs) - min(1.0, n)) < 4e-3 * min(1.0, n), scale
    # one huge value among ordinary ones, and zeros
    g = torch.zeros(30000, device="cuda")
    assert float(ops.grad_norm([g])) == 0.0
    assert float(ops.clip_grad_norm([g], 1.0)) == 0.0 and not g.any()
    g[12345] = 3e30
    assert abs(float(ops.grad_norm([g])) - 3e30) < 1e24


def test_not_finite():
    for bad, want in ((float("inf"), math.inf), (float("nan"), math.nan)):
        gs = tensors([9000, 100], seed=2)
        gs[1][50] = bad
        outs = [torch.empty_like(g) for g in gs]
        n = float(ops.clip_grad_norm(gs, 1.0, outs=outs))
        if math.isinf(want):   # scale 0: finite values vanish, infinity times 0 is NaN
            assert math.isinf(n) and not outs[0].any() and torch.isnan(outs[1][50]) and not outs[1][:50].any()
        else:
            assert math.isnan(n) and all(torch.isnan(o).all() for o in outs)


def test_max_norm_zero_and_repeats():
    gs = tensors([70000, 33], seed=3)
    outs = [torch.empty_like(g) for g in gs]
    ops.clip_grad_norm(gs, 0.0, outs=outs)
    assert not any(o.any() for o in outs)
    a, b = ops.grad_norm(gs), ops.grad_norm(gs)
    assert torch.equal(a, b)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        c = ops.grad_norm(gs)
    side.synchronize()
    assert torch.equal(a, c)


def test_no_tensors():
    n = torch.full((1,), 9.0, device="cuda")
    assert float(ops.clip_grad_norm([], 1.0, norm=n)) == 0.0
    assert float(ops.grad_norm([torch.empty(0, device="cuda")])) == 0.0


def test_in_a_graph():
    gs = tensors([40000, 5], seed=4)
    outs = [torch.empty_like(g) for g in gs]
    norm, ws = torch.empty(1, device="cuda"), ops.Workspace()
    ops.clip_grad_norm(gs, 1.0, outs=outs, norm=norm, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.clip_grad_norm(gs, 1.0, outs=outs, norm=norm, workspace=ws)
    for g in gs:
        g.mul_(3.0)
    graph.replay()
    torch.cuda.synchronize()
    n = norm64(gs)
    assert abs(float(norm) - n) < 2e-7 * n
