"""The gated recurrent layer's operators together, as the example's model runs them: it
runs, its gradients are those of the same model in 64 bits, a step of it goes into a
CUDA graph, and its calls leave a busy current stream alone.

Tolerance of the gradients, in norm: activations and cotangents are rounded to bf16
after every operation, by at most 2^-8 of each value; from the loss to a weight of the
first block and back lie about a dozen of them, 12 2^-8 = 5e-2.
"""
import importlib.util
import os

import pytest
import torch

from preconditioned_delta_rule_phase1_gb300 import build as osdn_build
from preconditioned_delta_rule_phase1_gb300 import ops

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    osdn_build.build()
    spec = importlib.util.spec_from_file_location("recurrent_layer", os.path.join(ROOT, "examples", "recurrent_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_runs(m):
    off, loss, status = m.main()
    assert status == 0 and all(map(lambda v: v == v, loss))
    # two ways of rounding the same bf16 activations, a few operations deep
    assert off < 5e-2


def model64(w, x, first, padded, states):
    """The example's forward pass in 64 bits, by autograd's operations."""
    out, s = None, x
    for i, p in enumerate(w):
        s = x if out is None else s + out
        mean = s.mean(-1, keepdim=True)
        y = (s - mean) / ((s - mean).square().mean(-1, keepdim=True) + 1e-5).sqrt() * p["weight"] + p["bias"]
        xs, gate = y @ p["x"], y @ p["gate"] + p["memory"]
        a = torch.sigmoid(gate)
        # (a derivative of the root at a = 1 does not exist: padding is put in afterwards)
        wx = ((1 - a) * (1 + a)).sqrt() * xs
        h, all_h = states[i], []
        for t in range(x.shape[1]):
            kept = torch.where(first[:, t, None], torch.zeros_like(h), a[:, t] * h)
            new = torch.where(first[:, t, None], xs[:, t], kept + wx[:, t])
            h = torch.where(padded[:, t, None], h, new)
            all_h.append(h)
        out = torch.stack(all_h, 1) @ p["out"]
    return s + out


def test_gradients_of_the_example(m):
    model = m.Model(seed=3)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(2, 90, m.WIDTH, generator=g, device="cuda").bfloat16()
    states = [torch.randn(2, m.CHANNELS, generator=g, device="cuda") for _ in range(m.BLOCKS)]
    first, padded = (torch.zeros(2, 90, dtype=torch.bool, device="cuda") for _ in range(2))
    first[:, 31], padded[1, 70:] = True, True
    dout = torch.randn(2, 90, m.WIDTH, generator=g, device="cuda").bfloat16().masked_fill(padded[..., None], 0)
    out, _, saved = model.prompt(x, states, first, padded)
    grads, dx = model.gradients(saved, dout)
    w = [{n: t.double().requires_grad_() for n, t in b.items()} for b in model.w]
    x64 = x.double().requires_grad_()
    ref = model64(w, x64, first, padded, [s.double() for s in states])
    names = [(i, n) for i, b in enumerate(w) for n in b]
    want = torch.autograd.grad((ref * dout.double()).sum(), [w[i][n] for i, n in names] + [x64])
    off = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    assert off(out.masked_fill(padded[..., None], 0), ref.detach().masked_fill(padded[..., None], 0)) < 5e-2
    for (i, n), v in zip(names, want):
        assert off(grads[i][n], v) < 5e-2, (i, n)
    assert off(dx, want[-1]) < 5e-2


def test_a_step_in_a_graph(m):
    model = m.Model(seed=4)
    x = torch.randn(2, 200, m.WIDTH, device="cuda").bfloat16()
    dout = torch.randn_like(x)
    token = torch.randn(2, m.WIDTH, device="cuda").bfloat16()

    def run():
        out, ends, saved = model.prompt(x)
        grads, dx = model.gradients(saved, dout)
        return [out, model.token(token, ends), dx] + [v for b in grads for v in b.values()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(2):
        x.mul_(-1.25)
        graph.replay()
        torch.cuda.synchronize()
        want = run()
        for a, b in zip(got, want):   # (the products around the calls may take another route in a graph)
            assert float((a.double() - b.double()).norm() / b.double().norm()) < 2e-2


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("grow", [False, True])
def test_a_busy_current_stream_is_no_part_of_the_call(m, io, grow):
    x, gate, dh = (torch.randn(2, 3000, 130, device="cuda").to(io) for _ in range(3))
    h0, w = torch.randn(2, 130, device="cuda"), torch.randn(130, device="cuda")
    h, _ = ops.gated_scan(x, gate, h0)
    calls = {
        "gated_scan": lambda **k: ops.gated_scan(x, gate, h0, **k),
        "gated_scan_backward": lambda **k: list(ops.gated_scan_backward(x, gate, h, h0, dh=dh, **k).values()),
        "layer_norm": lambda workspace=None, **k: ops.layer_norm(x, w, w, residual=gate, **k),
        "layer_norm_backward": lambda **k: list(ops.layer_norm_backward(x, dh, w, w, ds=gate, **k).values()),
    }
    a = torch.randn(8192, 8192, device="cuda")
    side = torch.cuda.Stream()
    for name, call in calls.items():
        want = call()
        with torch.cuda.stream(side):   # everything loaded and allocated once
            call()
        ws = ops.Workspace(stream=side) if grow else None
        torch.cuda.synchronize()
        for _ in range(30):
            a @ a   # half a second of the current stream or so
        busy = torch.cuda.Event()
        busy.record()
        got = call(stream=side, workspace=ws)
        # what the call has freed is not handed to the current stream
        junk = [torch.full((n,), 0xff, dtype=torch.uint8, device="cuda") for n in (4096, 1 << 20, 1 << 23)]
        done = torch.cuda.Event()
        done.record(side)
        done.synchronize()
        assert not busy.query(), name   # the call did not wait for the current stream
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want)), name
        del junk
