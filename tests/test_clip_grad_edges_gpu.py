"""Global gradient norm and clipping at the edges of its tables of tensors.

Tolerance of the norm 2e-7, as for every other size: the sum keeps its
rounding errors and is rounded to fp32 once.
"""
import pytest
import torch

from preconditioned_delta_rule_phase1_gb300 import build as osdn_build
from preconditioned_delta_rule_phase1_gb300 import ops
from tests.test_clip_grad_gpu import norm64, tensors

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    osdn_build.build()
    ops.lib()


@pytest.mark.parametrize("sizes", [[5] * 1024 + [0], [5] * 1024 + [0] * 2000, [0] * 30 + [7] * 1024 + [0, 0],
                                   [5] * 1023 + [0, 0], [5] * 1024 + [0, 9], [0] * 1500 + [3], [5] * 2048 + [0],
                                   [5] * 47 + [0], [5] * 48 + [0]],
                         ids=lambda s: "%d tensors, %d empty" % (len(s), s.count(0)))
def test_full_tables_and_empty_tensors(sizes):
    gs = tensors(sizes, seed=len(sizes))
    n = norm64(gs)
    norm = torch.full((1,), 123.0, device="cuda")
    assert abs(float(ops.grad_norm(gs, norm=norm)) - n) < 2e-7 * n
    outs = [torch.full_like(g, 5.0) for g in gs]
    norm.fill_(123.0)
    ops.clip_grad_norm(gs, 0.25 * n, outs=outs, norm=norm)
    assert abs(float(norm) - n) < 2e-7 * n
    for g, o in zip(gs, outs):   # the scale and the product round once each
        ulp = 2.0 ** -8 if g.dtype == torch.bfloat16 else 2.0 ** -22
        want = g.double() * 0.25
        assert ((o.double() - want).abs() <= ulp * want.abs()).all()
    inplace = [g.clone() for g in gs]
    norm.fill_(123.0)
    ops.clip_grad_norm(inplace, 0.25 * n, norm=norm)
    assert abs(float(norm) - n) < 2e-7 * n
    assert all(torch.equal(a, b) for a, b in zip(inplace, outs))


def test_a_tensor_counted_twice():
    # tied weights: the norm alone writes nothing
    gs = tensors([5000, 300], seed=9)
    n = norm64([gs[0], *gs])
    assert abs(float(ops.grad_norm([gs[0], *gs])) - n) < 2e-7 * n
    # two outputs that share elements
    out = torch.empty_like(gs[0])
    with pytest.raises(ops.OsdnError, match="overlaps"):
        ops.clip_grad_norm(gs, 1.0, outs=[out, out.view(torch.bfloat16)[8:308]])
