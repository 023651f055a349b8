"""What the binding of the decayed layer's calls does before a call, on the
CPU: tensors and the library are stand-ins."""
import contextlib

import pytest
import torch

from preconditioned_delta_rule_phase1_gb300 import ops


class Fake:
    """As much of a CUDA tensor as the binding looks at."""

    def __init__(self, device, *shape, dtype=torch.float32):
        self.device, self.shape, self.dtype = torch.device("cuda", device), torch.Size(shape), dtype

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20

    def numel(self):
        return self.shape.numel()


class FakeWorkspace:
    def __init__(self, device):
        self.buf = Fake(device, 256)

    def ensure(self, n):
        self.buf.shape = torch.Size((n,))


@pytest.fixture
def device(monkeypatch):
    """The current device, as a list of one number."""
    now = [0]

    @contextlib.contextmanager
    def use(d):
        before, now[0] = now[0], d.index
        yield
        now[0] = before
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: type("S", (), {"cuda_stream": 0}))
    return now


def test_workspace_sizes_are_those_of_the_tensors_device(monkeypatch, device):
    # a device with more SMs cuts the time axis into more ranges: its calls need more workspace
    need, given = {0: 1000, 1: 5000, 2: 3000}, []

    class Lib:
        def osdn_decay_attn_workspace_bytes(self, *shape):
            return need[device[0]]

        def osdn_decay_attn(self, *args):
            given.append((device[0], args[-2]))
            return 0
    lib = Lib()
    monkeypatch.setattr(ops, "lib", lambda: lib)
    monkeypatch.setattr(ops, "_lib", lib)
    for d in (0, 1, 2, 0, 1):
        # a shape that no other test asks for
        q, k, v, o = (Fake(d, 1, 1, 77777, 64) for _ in range(4))
        ops.decay_attn(q, k, v, Fake(d, 1), o=o, ST=Fake(d, 1, 1, 64, 64), workspace=FakeWorkspace(d))
    assert given == [(d, need[d]) for d in (0, 1, 2, 0, 1)]


def test_a_tensor_may_be_counted_twice_but_not_written_twice():
    g = torch.zeros(40)
    with pytest.raises(ValueError, match="CUDA tensors only"):   # no argument was refused
        ops.grad_norm([g, g])
    with pytest.raises(ValueError, match="written twice"):
        ops.clip_grad_norm([g, g], 1.0)
    with pytest.raises(ValueError, match="written twice"):
        ops.clip_grad_norm([g, torch.zeros(40)], float("inf"), outs=[g, g])
