"""Calls with ``stream=`` and no workspace, or one that has to grow, while the
current stream is busy: nothing of the call waits for the current stream, or
is left to it, so the results are those of an ordinary call."""
import pytest
import torch

from preconditioned_delta_rule_phase1_gb300 import build as osdn_build
from preconditioned_delta_rule_phase1_gb300 import ops, synth
from tests._util import to_cuda
from tests.test_decay_attn_gpu import inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    osdn_build.build()
    ops.lib()


def calls(io):
    # shapes that the attention cuts into ranges: the workspace holds their states
    x = inputs(1, 4, 3000, 128, 128, io, seed=8, decay=torch.tensor([0.99, 0.999, 1.0, 0.9]))
    w, gate, dy = (torch.randn(*s, device="cuda") for s in ((512,), (1, 3000, 512), (1, 3000, 512)))
    gate, dy = gate.to(x["q"].dtype), dy.to(x["q"].dtype)
    qkv = (x["q"], x["k"], x["v"])
    g = to_cuda(synth.make_random(1, 2, 700, 128, 128, io=io, apf=True, gated=True, s0=True, seed=3))
    return {
        "decay_attn": lambda **k: ops.decay_attn(*qkv, x["decay"], x["S0"], **k),
        "decay_attn_backward": lambda **k: ops.decay_attn_backward(*qkv, x["decay"], x["S0"], do=x["do"],
                                                                   dST=x["dST"], **k),
        "group_norm_backward": lambda **k: ops.group_norm_backward(x["v"], dy, w, w, gate, act="silu", **k),
        "clip_grad_norm": lambda **k: ops.clip_grad_norm(list(qkv), float("inf"), **k),
        "forward": lambda **k: ops.forward(g["q"], g["k"], g["v"], g["beta"], g["r"], g["eta"], g["d0"], g["alpha"],
                                           g["S0"], **k),
    }


def flat(out):
    return [out] if isinstance(out, torch.Tensor) else list(out.values()) if isinstance(out, dict) else list(out)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("grow", [False, True])
def test_a_busy_current_stream_is_no_part_of_the_call(io, grow):
    a = torch.randn(8192, 8192, device="cuda")
    side = torch.cuda.Stream()
    for name, call in calls(io).items():
        want = flat(call())
        with torch.cuda.stream(side):   # everything loaded and allocated once
            call()
        ws = ops.Workspace(stream=side) if grow else None
        torch.cuda.synchronize()
        for _ in range(30):
            a @ a   # half a second of the current stream or so
        busy = torch.cuda.Event()
        busy.record()
        got = flat(call(stream=side, workspace=ws))
        # what the call has freed is not handed to the current stream
        junk = [torch.full((n,), 0xff, dtype=torch.uint8, device="cuda") for n in (4096, 1 << 20, 1 << 23)]
        done = torch.cuda.Event()
        done.record(side)
        done.synchronize()
        assert not busy.query(), name   # the call did not wait for the current stream
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)), name
        assert ws is None or ws.status() == 0
        del junk
