"""A call with ``stream=`` allocates, grows its workspace and launches under
that stream, on the CPU: the library is a stand-in and torch's current stream
a variable, which every allocation and launch of a call is noted with."""
import contextlib
import ctypes

import pytest
import torch

from preconditioned_delta_rule_phase1_gb300 import ops, synth

SIDE = "side"


@pytest.fixture
def seen(monkeypatch):
    """(what, stream) of every allocation and launch since the test began."""
    now, notes = ["current"], []

    @contextlib.contextmanager
    def use(stream):
        before, now[0] = now[0], stream
        yield
        now[0] = before

    def note(what, fn):
        def call(*args, **kw):
            notes.append((what, now[0]))
            return fn(*args, **kw)
        return call

    class Lib:
        def __getattr__(self, name):
            if name.endswith("workspace_bytes"):
                return lambda *a: 4096
            return note(name, lambda *a: 0)

    for name in ("empty", "empty_like", "zeros"):
        monkeypatch.setattr(torch, name, note(name, getattr(torch, name)))
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(ops, "lib", lambda: Lib())
    monkeypatch.setattr(ops, "_lib", Lib())
    monkeypatch.setattr(ops, "_on", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(ops, "_stream", lambda stream, device=None: ctypes.c_void_p(0))
    monkeypatch.setattr(ops, "_ptr", lambda t: None)

    def run(name, device, stream, args, workspace=None, *size):
        if workspace is not None:
            workspace.ensure(4096)
        notes.append((name, now[0]))
    monkeypatch.setattr(ops, "_run", run)
    return notes


def calls():
    x = synth.make_random(1, 2, 5, 64, 64, io="f32", apf=True, gated=True, s0=True, d0=True)
    a, one = torch.rand(2), {n: x[n][:, :, 0].contiguous() for n in ("q", "k", "v", "beta")}
    ak, kt = torch.rand(1, 2, 5, 64), torch.rand(1, 2, 5, 64)
    d, S, do = torch.rand(1, 2, 64), torch.rand(1, 2, 64, 64), torch.rand(1, 2, 5, 64)
    y = torch.rand(1, 5, 128)
    qkv, tok = (x["q"], x["k"], x["v"]), (one["q"], one["k"], one["v"])
    return {
        "precond_scan": lambda s: ops.precond_scan(x["k"], x["beta"], stream=s),
        "precond_scan residual": lambda s: ops.precond_scan(x["k"], x["beta"], log_ratio=True, stream=s),
        "precond_scan_noalloc": lambda s: ops.precond_scan_noalloc(x["k"], x["beta"], stream=s),
        "chunk_fwd": lambda s: ops.chunk_fwd(x["q"], x["k"], kt, x["v"], x["beta"], stream=s),
        "forward": lambda s: ops.forward(*qkv, x["beta"], stream=s),
        "forward_fused": lambda s: ops.forward_fused(*qkv, x["beta"], stream=s),
        "decode_step": lambda s: ops.decode_step(*tok, one["beta"], d, S, stream=s),
        "decode_step_kda": lambda s: ops.decode_step_kda(*tok, one["beta"], d, S, stream=s),
        "backward": lambda s: ops.backward(x["q"], x["k"], kt, x["v"], x["beta"], do=do, stream=s),
        "backward_kda": lambda s: ops.backward_kda(x["q"], x["k"], kt, x["v"], x["beta"], alpha_k=ak, do=do, stream=s),
        "chunk_fwd_kda": lambda s: ops.chunk_fwd_kda(x["q"], x["k"], kt, x["v"], x["beta"], ak, stream=s),
        "forward_kda": lambda s: ops.forward_kda(*qkv, x["beta"], alpha_k=ak, stream=s),
        "decay_attn": lambda s: ops.decay_attn(*qkv, a, stream=s),
        "decay_attn by position": lambda s: ops.decay_attn(*qkv, a, None, None, None, None, s),
        "decay_attn_step": lambda s: ops.decay_attn_step(*tok, a, S, stream=s),
        "decay_attn_backward": lambda s: ops.decay_attn_backward(*qkv, a, x["S0"], do=do, stream=s),
        "group_norm": lambda s: ops.group_norm(x["v"], stream=s),
        "group_norm_backward": lambda s: ops.group_norm_backward(x["v"], y, stream=s),
        "clip_grad_norm": lambda s: ops.clip_grad_norm([d, S], 1.0, stream=s),
        "grad_norm": lambda s: ops.grad_norm([d, S], stream=s),
    }


@pytest.mark.parametrize("name", sorted(calls()))
def test_everything_happens_on_the_stream(seen, name):
    call = calls()[name]
    seen.clear()
    call(SIDE)
    assert any(w.startswith("osdn_") for w, _ in seen) and any(not w.startswith("osdn_") for w, _ in seen)
    assert not [w for w, stream in seen if stream != SIDE]
    seen.clear()
    call(None)
    assert seen and not [w for w, stream in seen if stream != "current"]


def test_a_workspace_is_made_and_grown_on_its_stream(seen):
    ws = ops.Workspace(device="cpu", stream=SIDE)
    ws.ensure(10000, SIDE)
    assert [s for w, s in seen if w == "zeros"] == [SIDE, SIDE] and ws.nbytes >= 10000
    ws.ensure(20000)
    assert seen[-1] == ("zeros", "current")


def test_a_stream_of_another_device_is_refused():
    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 0
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        ops._stream(Stream(), torch.device("cuda", 0))
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        ops._run("osdn_group_norm", torch.device("cuda", 0), Stream(), ())
