"""Layer norm and its gradients at rows whose first value lies far from the others, and
at sizes where squares or cubes of what is formed on the way could leave fp32, element
by element against the formula in 64 bits.

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


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("C", [40, 255, 513, 1000, 2047, 2048, 5000, 8192, 16383, 16384])
def test_the_others_keep_their_digits(io, C):
    g = torch.Generator().manual_seed(C)
    x, dy = torch.randn(10, C, generator=g), torch.randn(10, C, generator=g)
    x += 0.3
    for r, far in enumerate((0.0, 5.0, 30.0, -300.0, 3e3, -1e5, 1e6, -1e7, 1e4, 100.0)):
        x[r, 0] += far
    x[8, C // 2] = -1e4   # another one far out, where the sums do not begin
    check(x.to(DT[io]).cuda(), dy.to(DT[io]).cuda(), io, 1e-5, C)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,C", [(3, 2048), (1500, 2048), (1500, 690), (1500, 300)])
def test_the_sum_with_a_residual(residual, rows, C):
    """The same with what few and many rows choose, and for the sum's norm."""
    g = torch.Generator().manual_seed(C)
    x, res = torch.randn(rows, C, generator=g), torch.randn(rows, C, generator=g)
    x[::3, 0] = 2e5
    x, res = x.cuda(), res.cuda()
    s = x + res if residual else x
    d = s.double() - mean(s.double())
    xh = d / (mean(d * d) + 1e-5).sqrt()
    y = ops.layer_norm(x, residual=res)[0] if residual else ops.layer_norm(x)
    tol = 48 * U * mean(xh.abs()) + 60 * U * xh.abs()
    assert bool(((y.double() - xh).abs() <= tol).all())


@pytest.mark.parametrize("C", [64, 1000, 2048, 5000, 16384])
@pytest.mark.parametrize("size,grad", [(1e16, 1e-3), (3e15, 1e-12), (1e-12, 1.0), (1e-17, 1e-3), (1.0, 1e-30)])
def test_sizes_at_the_ends(C, size, grad):
    """dx is about grad / size (what of it is below fp32's normal range is not looked at)."""
    g = torch.Generator().manual_seed(C)
    x = (size * (0.3 + torch.randn(6, C, generator=g))).cuda()
    dy = (grad * torch.randn(6, C, generator=g)).cuda()
    check(x, dy, "f32", 1e-36, (C, size, grad))
