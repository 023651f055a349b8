"""The gated recurrent layer's calls with ``stream=`` allocate, grow their
workspace and launch under that stream (the library is a stand-in, as for the
other calls)."""
import pytest
import torch

from preconditioned_delta_rule_phase1_gb300 import ops
from tests.test_streams_cpu import SIDE, seen  # noqa: F401


def calls():
    x, h0, w = torch.rand(2, 5, 64), torch.rand(2, 64), torch.rand(64)
    return {
        "gated_scan": lambda s: ops.gated_scan(x, x, h0, stream=s),
        "gated_scan by position": lambda s: ops.gated_scan(x, x, h0, "unit", None, None, None, s),
        "gated_scan_step": lambda s: ops.gated_scan_step(h0, h0, h0, stream=s),
        "gated_scan_backward": lambda s: ops.gated_scan_backward(x, x, x, h0, dh=x, stream=s),
        "layer_norm": lambda s: ops.layer_norm(x, w, w, residual=x, stream=s),
        "layer_norm_backward": lambda s: ops.layer_norm_backward(x, x, w, w, stream=s),
    }


@pytest.mark.parametrize("name", sorted(calls()))
def test_everything_happens_on_the_stream(seen, name):  # noqa: F811
    call = calls()[name]
    seen.clear()
    call(SIDE)
    assert any(w.startswith("osdn_") for w, _ in seen) and any(not w.startswith("osdn_") for w, _ in seen)
    assert not [w for w, stream in seen if stream != SIDE]
    seen.clear()
    call(None)
    assert seen and not [w for w, stream in seen if stream != "current"]
