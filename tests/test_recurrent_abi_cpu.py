"""The gated recurrent layer's calls refuse bad arguments on the host, before
anything is enqueued, and the binding refuses tensors that do not fit (no GPU
needed)."""
import pytest
import torch

from preconditioned_delta_rule_phase1_gb300 import build as osdn_build
from preconditioned_delta_rule_phase1_gb300 import ops

F = 0x100000   # never dereferenced: every case fails validation first
FINE = (-6, -10)   # no argument was refused: it got as far as the device check


@pytest.fixture(scope="module")
def L():
    osdn_build.build()
    return ops.lib()


def test_gated_scan(L):
    def scan(io=1, B=1, T=8, C=64, mix=1, x=F, gate=2 * F, h0=3 * F, h=4 * F, hT=5 * F):
        return L.osdn_gated_scan(io, B, T, C, mix, x, gate, h0, h, hT, None)
    assert scan(io=2) == -3 and scan(io=-1) == -3
    assert scan(B=-1) == -2 and scan(T=-1) == -2 and scan(C=-1) == -2
    assert scan(T=1073741761) == -2 and scan(C=(1 << 24) + 1) == -2
    assert scan(B=1 << 20, T=1 << 20) == -2 and scan(B=2147483647, C=64) == -2
    assert scan(mix=3) == -12 and scan(mix=-1) == -12
    for n in ("x", "gate", "h"):
        assert scan(**{n: None}) == -1, n
    for n in ("x", "gate", "h0", "h", "hT"):
        assert scan(**{n: 9 * F + 4}) == -4, n
    for n in ("x", "gate", "h0"):
        assert scan(**{n: 4 * F + 16}) == -9 and scan(**{n: 5 * F + 16}) == -9, n
    assert scan(hT=4 * F) == -9 and scan(h=5 * F - 1008) == -9 and scan(h=5 * F - 1024) in FINE
    assert scan(x=F, gate=F) in FINE and scan(h0=None, hT=None) in FINE
    assert scan(B=0) == 0 and scan(C=0) == 0 and scan(B=0, x=None, gate=None, h=None) == 0
    assert scan(T=0, x=None, gate=None, h=None) in FINE


def test_gated_scan_step(L):
    def step(io=1, B=1, C=64, mix=1, x=F, gate=2 * F, h=3 * F, y=4 * F):
        return L.osdn_gated_scan_step(io, B, C, mix, x, gate, h, y, None)
    assert step(io=7) == -3 and step(B=-1) == -2 and step(C=-5) == -2 and step(mix=9) == -12
    assert step(B=1 << 30, C=1 << 10) == -2
    for n in ("x", "gate", "h", "y"):
        assert step(**{n: None}) == -1 and step(**{n: 9 * F + 8}) == -4, n
    assert step(y=F) == -9 and step(h=F) == -9 and step(gate=3 * F) == -9 and step(y=3 * F) == -9
    assert step(B=0) == 0 and step() in FINE


def test_gated_scan_backward(L):
    names = ["x", "gate", "h", "h0", "d_h", "d_hT", "dx", "dgate", "dh0"]

    def back(io=1, B=1, T=8, C=64, mix=1, **kw):
        at = {n: (i + 1) * F for i, n in enumerate(names)}
        at.update(kw)
        return L.osdn_gated_scan_backward(io, B, T, C, mix, *[at[n] for n in names], None)
    assert back(io=5) == -3 and back(T=-3) == -2 and back(mix=4) == -12
    for n in ("x", "gate", "h", "d_h", "dx", "dgate"):
        assert back(**{n: None}) == -1, n
    for n in names:
        assert back(**{n: 20 * F + 2}) == -4, n
    for n in ("dx", "dgate", "dh0"):
        for other in names:
            if other != n:
                assert back(**{n: names.index(other) * F + F}) == -9, (n, other)
    assert back(h0=None, d_hT=None, dh0=None) in FINE and back(B=0) == 0


def test_layer_norm(L):
    def norm(io=1, rows=3, C=64, x=F, res=None, w=2 * F, b=3 * F, eps=1e-5, y=4 * F, s=None):
        return L.osdn_layer_norm(io, rows, C, x, res, w, b, eps, y, s, None)
    assert norm(io=3) == -3
    assert norm(C=0) == -2 and norm(C=16385) == -2 and norm(rows=-1) == -2 and norm(rows=1 << 31) == -2
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert norm(eps=eps) == -12
    assert norm(x=None) == -1 and norm(y=None) == -1
    assert norm(res=5 * F) == -1 and norm(s=5 * F) == -1   # a sum exactly with a residual
    for n in ("x", "w", "b", "y"):
        assert norm(**{n: 9 * F + 8}) == -4, n
    assert norm(y=F) == -9 and norm(w=4 * F) == -9 and norm(res=4 * F, s=6 * F) == -9
    assert norm(res=5 * F, s=F) == -9 and norm(res=5 * F, s=4 * F) == -9 and norm(res=F, s=6 * F) in FINE
    assert norm(rows=0) == 0 and norm() in FINE


def test_layer_norm_backward(L):
    names, outs = ["x", "dy", "w", "ds"], ["dx", "dw", "db", "ws"]

    def back(io=1, rows=3, C=64, eps=1e-5, wsb=None, **kw):
        at = {n: (i + 1) * F for i, n in enumerate(names + outs)}
        at.update(kw)
        wsb = L.osdn_layer_norm_backward_workspace_bytes(rows, C) if wsb is None else wsb
        return L.osdn_layer_norm_backward(io, rows, C, at["x"], at["dy"], at["w"], at["ds"], eps,
                                          *[at[n] for n in outs], wsb, None)
    assert back(io=3) == -3 and back(C=20000, wsb=1 << 30) == -2 and back(eps=0.0) == -12
    assert back(wsb=256) == -5 and back(ws=None) == -5
    for n in ("x", "dy", "dx"):
        assert back(**{n: None}) == -1, n
    for n in names + outs:
        assert back(**{n: 20 * F + 4}) == -4, n
    for n in outs:
        assert back(**{n: 2 * F}) == -9, n
    assert back(w=None, ds=None, dw=None, db=None) in FINE
    assert L.osdn_layer_norm_backward_workspace_bytes(-1, 64) == 256
    # a share of both sums for every CTA that runs, whatever the number of rows
    for C in (1, 500, 8192, 16384):
        assert 256 < L.osdn_layer_norm_backward_workspace_bytes(1 << 20, C) <= 256 + 1024 * C * 8


def test_binding_refusals():
    c = torch.zeros
    x, h0 = c(2, 5, 64), c(2, 64)
    with pytest.raises(ValueError, match="CUDA tensors only"):   # no argument was refused
        ops.gated_scan(x, x, h0)
    with pytest.raises(ValueError, match="mix"):
        ops.gated_scan(x, x, mix="max")
    with pytest.raises(ValueError, match="gate has shape"):
        ops.gated_scan(x, x[:, :4])
    with pytest.raises(TypeError, match="gate has dtype"):
        ops.gated_scan(x, x.bfloat16())
    with pytest.raises(TypeError, match="h0 has dtype"):
        ops.gated_scan(x.bfloat16(), x.bfloat16(), h0.bfloat16())
    with pytest.raises(ValueError, match="contiguous"):
        ops.gated_scan(c(2, 64, 5).transpose(1, 2), x)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        ops.gated_scan(x.half(), x.half())
    with pytest.raises(ValueError, match="hT has shape"):
        ops.gated_scan(x, x, hT=c(64))
    with pytest.raises(ValueError, match="h has shape"):
        ops.gated_scan_step(h0, h0, c(2, 65))
    with pytest.raises(TypeError, match="h has dtype"):
        ops.gated_scan_step(h0.bfloat16(), h0.bfloat16(), h0.bfloat16())
    with pytest.raises(TypeError, match="dh has dtype"):
        ops.gated_scan_backward(x, x, x, dh=x.bfloat16())
    with pytest.raises(ValueError, match="dhT has shape"):
        ops.gated_scan_backward(x, x, x, dh=x, dhT=c(2, 1, 64))
    w = c(64)
    with pytest.raises(ValueError, match="CUDA tensors only"):
        ops.layer_norm(x, w, w, residual=x)
    with pytest.raises(ValueError, match="weight has shape"):
        ops.layer_norm(x, c(5))
    with pytest.raises(TypeError, match="bias has dtype"):
        ops.layer_norm(x, w, w.bfloat16())
    with pytest.raises(ValueError, match="residual has shape"):
        ops.layer_norm(x, residual=x[:1])
    with pytest.raises(ValueError, match="there is none"):
        ops.layer_norm(x, s=x)
    with pytest.raises(ValueError, match="last dimension"):
        ops.layer_norm(torch.tensor(1.0))
    with pytest.raises(ValueError, match="dy has shape"):
        ops.layer_norm_backward(x, x[:1])
    with pytest.raises(TypeError, match="ds has dtype"):
        ops.layer_norm_backward(x, x, ds=x.bfloat16())
    with pytest.raises(ValueError, match="bias has shape"):
        ops.layer_norm_backward(x, x, bias=c(65))
