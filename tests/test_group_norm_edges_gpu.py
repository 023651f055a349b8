"""The group norm and its gradients captured into a CUDA graph."""
import pytest
import torch

from preconditioned_delta_rule_phase1_gb300 import build as osdn_build
from preconditioned_delta_rule_phase1_gb300 import ops
from tests.test_group_norm_gpu import inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    osdn_build.build()
    ops.lib()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("first", [False, True])
def test_in_a_graph(io, first):
    t = inputs(2, 4, 77, 128, io, first, True, True, seed=4)
    kw = dict(groups=4, act="silu")
    ws = ops.Workspace()
    fwd = lambda: ops.group_norm(t["x"], t["weight"], t["bias"], t["gate"], **kw)  # noqa: E731
    bwd = lambda: ops.group_norm_backward(t["x"], t["dy"], t["weight"], t["bias"], t["gate"], workspace=ws,  # noqa: E731
                                          **kw)
    fwd(), bwd()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, g = fwd(), bwd()
    t["x"].mul_(-2.0)
    t["dy"].add_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    want = bwd()
    assert torch.equal(y, fwd()) and all(torch.equal(g[n], want[n]) for n in want)
