"""Layer norm and its gradients at sizes where squares or cubes of what is formed on the
way could leave fp32, element by element against the formula in 64 bits.

Tolerance.  A row's mean is a sum of at most 48 roundings one after the other (32 values
of a thread in pairs, 5 exchanges, 16 warps, and those of the differences), so it is off
by at most 48 2^-24 of the mean size of the differences to it, and so is every
difference, beside 8 roundings of its own size.  The variance and the mean products are
off by as much of theirs.  Then half a step of the I/O type.
"""
import pytest
import torch

from preconditioned_delta_rule_phase1_gb300 import build as osdn_build
from preconditioned_delta_rule_phase1_gb300 import ops

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    osdn_build.build()
    ops.lib()


def mean(v):
    return v.mean(-1, keepdim=True)


def check(x, dy, io, eps, what):
    s, u = x.double(), dy.double()
    d = s - mean(s)
    r = 1 / (mean(d * d) + eps).sqrt()
    xh = d * r
    off = 48 * U * mean(xh.abs()) + 56 * U * xh.abs()   # of a normed value
    y = ops.layer_norm(x, eps=eps)
    bad = (y.double() - xh).abs() - (HALF[io] * xh.abs() + off)
    assert bool((bad <= 0).all()), ("y", what, float(bad.max()))
    c = mean(u * xh)
    dx = r * (u - mean(u) - xh * c)
    got = ops.layer_norm_backward(x, dy, eps=eps)["x"].double()
    tol = r * (48 * U * mean(u.abs()) + 8 * U * u.abs() + off * c.abs()
               + xh.abs() * (56 * U * mean((u * xh).abs()) + mean(u.abs() * off))) + 56 * U * dx.abs()
    bad = (got - dx).abs() - (HALF[io] * dx.abs() + tol)
    assert bool((bad <= 0).all()), ("dx", what, float((bad / tol).max()))


@pytest.mark.parametrize("C", [64, 1000, 2048, 5000, 16384])
@pytest.mark.parametrize("size,grad", [(1e16, 1e-3), (3e15, 1e-12), (1e-12, 1.0), (1e-17, 1e-3), (1.0, 1e-30)])
def test_sizes_at_the_ends(C, size, grad):
    """dx is about grad / size (what of it is below fp32's normal range is not looked at)."""
    g = torch.Generator().manual_seed(C)
    x = (size * (0.3 + torch.randn(6, C, generator=g))).cuda()
    dy = (grad * torch.randn(6, C, generator=g)).cuda()
    check(x, dy, "f32", 1e-36, (C, size, grad))
