"""The decayed layer's calls refuse bad arguments on the host, before anything
is enqueued, and the binding refuses tensors that do not fit (no GPU needed)."""
import ctypes

import pytest
import torch

from preconditioned_delta_rule_phase1_gb300 import build as osdn_build
from preconditioned_delta_rule_phase1_gb300 import ops

F = 0x100000   # never dereferenced: every case fails validation first


@pytest.fixture(scope="module")
def L():
    osdn_build.build()
    return ops.lib()


def attn(L, io=1, B=1, H=1, T=8, K=64, V=64, q=F, k=2 * F, v=3 * F, decay=4 * F, S0=None, o=5 * F, ST=None,
         ws=6 * F, wsb=None):
    wsb = L.osdn_decay_attn_workspace_bytes(io, B, H, T, K, V) if wsb is None else wsb
    return L.osdn_decay_attn(io, B, H, T, K, V, q, k, v, decay, S0, o, ST, ws, wsb, None)


def test_decay_attn(L):
    assert attn(L, io=2) == -3
    assert attn(L, K=96) == -2 and attn(L, V=32) == -2 and attn(L, T=-1) == -2 and attn(L, B=4096, H=4097) == -2
    assert attn(L, T=1073741761, wsb=1 << 62) == -2
    assert attn(L, ws=None) == -5 and attn(L, wsb=255) == -5
    for n in ("q", "k", "v", "decay", "o"):
        assert attn(L, **{n: None}) == -1, n
    for n in ("q", "k", "v", "decay", "S0", "o", "ST", "ws"):
        assert attn(L, **{n: 9 * F + 4}) == -4, n
    assert attn(L, o=F) == -9 and attn(L, ST=4 * F) == -9 and attn(L, ws=2 * F) == -9
    assert attn(L, o=7 * F, ST=7 * F) == -9 and attn(L, ws=5 * F - 128) == -9
    assert attn(L, q=F, k=F) in (-6, -10)   # inputs may coincide: it got as far as the device check
    assert attn(L, B=0) == 0


def test_decay_attn_workspace(L):
    assert L.osdn_decay_attn_workspace_bytes(1, 2, 3, 0, 64, 64) == 256
    assert L.osdn_decay_attn_workspace_bytes(9, 2, 3, 10, 64, 64) == 256
    # at most one state a range, and ranges are bounded whatever the length
    for io in (0, 1):
        for T in (1, 100, 65536, 1 << 28):
            assert 256 <= L.osdn_decay_attn_workspace_bytes(io, 1, 16, T, 128, 128) <= 256 + 1024 * 65536
    need = L.osdn_decay_attn_workspace_bytes(1, 1, 1, 65536, 128, 128)
    assert need > 256 and attn(L, T=65536, K=128, V=128, q=1 << 30, k=2 << 30, v=3 << 30, o=4 << 30,
                               wsb=need - 1) == -5


def test_decay_attn_step(L):
    def step(io=1, B=1, H=1, K=64, V=64, q=F, k=2 * F, v=3 * F, decay=4 * F, S=5 * F, o=6 * F, ws=7 * F, wsb=256):
        return L.osdn_decay_attn_step(io, B, H, K, V, q, k, v, decay, S, o, ws, wsb, None)
    assert step(io=-1) == -3 and step(K=0) == -2 and step(B=-1) == -2
    assert step(wsb=128) == -5 and step(ws=None) == -5
    for n in ("q", "k", "v", "decay", "S", "o"):
        assert step(**{n: None}) == -1 and step(**{n: 9 * F + 8}) == -4, n
    assert step(S=F) == -9 and step(o=3 * F) == -9 and step(o=5 * F) == -9 and step(ws=4 * F) == -9
    assert step(H=0) == 0


def test_decay_attn_backward(L):
    names = ["q", "k", "v", "decay", "S0", "d_o", "d_ST", "dq", "dk", "dv", "dS0", "ws"]

    def back(io=1, B=1, H=1, T=8, K=64, V=64, wsb=None, **kw):
        at = {n: (i + 1) * F for i, n in enumerate(names)}
        at.update(kw)
        wsb = L.osdn_decay_attn_backward_workspace_bytes(io, B, H, T, K, V) if wsb is None else wsb
        return L.osdn_decay_attn_backward(io, B, H, T, K, V, *[at[n] for n in names], wsb, None)
    assert back(io=5) == -3 and back(V=65) == -2 and back(T=-3) == -2 and back(wsb=0) == -5
    for n in ("q", "k", "v", "decay", "d_o", "dq", "dk", "dv"):
        assert back(**{n: None}) == -1, n
    for n in names:
        assert back(**{n: 20 * F + 2}) == -4, n
    for n in ("dq", "dk", "dv", "dS0", "ws"):
        assert back(**{n: 6 * F}) == -9, n
    assert back(dk=8 * F) == -9
    assert back(B=0) == 0


def test_group_norm(L):
    def norm(io=1, B=1, G=2, T=3, D=64, first=0, x=F, w=None, b=None, gate=None, act=0, eps=1e-5, y=2 * F):
        return L.osdn_group_norm(io, B, G, T, D, first, x, w, b, gate, act, eps, y, None)
    assert norm(io=3) == -3
    assert norm(D=12) == -2 and norm(D=0) == -2 and norm(D=520) == -2 and norm(G=0) == -2 and norm(T=-1) == -2
    assert norm(B=1 << 12, G=1 << 12, T=1 << 20) == -2
    assert norm(act=3) == -12 and norm(act=-1) == -12
    assert norm(eps=0.0) == -12 and norm(eps=-1.0) == -12
    assert norm(eps=float("nan")) == -12 and norm(eps=float("inf")) == -12
    assert norm(x=None) == -1 and norm(y=None) == -1
    assert norm(x=F + 8) == -4 and norm(w=4 * F + 4) == -4 and norm(gate=4 * F + 4) == -4
    assert norm(y=F) == -9 and norm(gate=2 * F) == -9 and norm(b=2 * F) == -9
    assert norm(T=0) == 0 and norm(B=0) == 0


def test_group_norm_backward(L):
    names = ["x", "dy", "w", "b", "gate"]
    outs = ["dx", "dgate", "dw", "db", "ws"]

    def back(io=1, B=1, G=2, T=3, D=64, act=1, eps=1e-5, wsb=None, **kw):
        at = {n: (i + 1) * F for i, n in enumerate(names + outs)}
        at.update(kw)
        wsb = L.osdn_group_norm_backward_workspace_bytes(B, G, T, D) if wsb is None else wsb
        return L.osdn_group_norm_backward(io, B, G, T, D, 0, *[at[n] for n in names], act, eps,
                                          *[at[n] for n in outs], wsb, None)
    assert back(io=3) == -3 and back(D=7) == -2 and back(act=9) == -12 and back(eps=0.0) == -12
    assert back(wsb=256) == -5 and back(ws=None) == -5
    for n in ("x", "dy", "dx", "dgate"):
        assert back(**{n: None}) == -1, n
    for n in names + outs:
        assert back(**{n: 20 * F + 4}) == -4, n
    for n in outs:
        assert back(**{n: 2 * F}) == -9, n


def test_clip_grad_norm(L):
    def clip(n=2, g=(F, 2 * F), o=(3 * F, 4 * F), sizes=(10, 20), ios=(0, 1), limit=1.0, norm=5 * F, ws=6 * F,
             wsb=None):
        P = ctypes.c_void_p * len(g)
        wsb = L.osdn_clip_grad_norm_workspace_bytes(n) if wsb is None else wsb
        return L.osdn_clip_grad_norm(n, P(*g), P(*o) if o else None, (ctypes.c_longlong * len(sizes))(*sizes),
                                     (ctypes.c_int * len(ios))(*ios), limit, norm, ws, wsb, None)
    assert clip(n=-1) == -2 and clip(sizes=(10, -1)) == -2 and clip(sizes=(10, (1 << 40) + 1)) == -2
    assert clip(ios=(0, 7)) == -3
    assert clip(limit=-1.0) == -12 and clip(limit=float("nan")) == -12
    assert clip(ws=None) == -5 and clip(wsb=300) == -5
    assert clip(g=(F, None)) == -1 and clip(o=(3 * F, None)) == -1
    assert clip(g=(F + 2, 2 * F)) == -4 and clip(o=(3 * F, 4 * F + 8)) == -4
    assert clip(norm=5 * F + 2) == -4 and clip(ws=6 * F + 8) == -4
    assert clip(o=(F + 16, 4 * F)) == -9       # an output inside its own input
    assert clip(norm=F) == -9                  # the norm inside a gradient that is still being read
    assert clip(norm=3 * F) == -9
    assert clip(ws=2 * F) == -9
    assert clip(o=None, norm=F) == -9
    assert clip() in (-6, -10)                 # fine but for the missing device


def test_binding_refusals():
    c = torch.zeros
    q, k, v, a = c(1, 2, 5, 64), c(1, 2, 5, 64), c(1, 2, 5, 64), c(2)
    with pytest.raises(ValueError):   # not on a CUDA device
        ops.decay_attn(q, k, v, a, workspace=None)
    with pytest.raises(ValueError, match="decay"):
        ops.decay_attn(q, k, v, c(3))
    with pytest.raises(TypeError, match="decay"):
        ops.decay_attn(q, k, v, a.double())
    with pytest.raises(ValueError, match="q has shape"):
        ops.decay_attn(q[:, :1], k, v, a)
    with pytest.raises(ValueError, match="contiguous"):
        ops.decay_attn(q, k, c(1, 5, 2, 64).transpose(1, 2), a)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        ops.decay_attn(q.half(), k.half(), v.half(), a)
    with pytest.raises(ValueError, match="S has shape"):
        ops.decay_attn_step(q[:, :, 0].contiguous(), k[:, :, 0].contiguous(), v[:, :, 0].contiguous(), a,
                            c(1, 2, 64, 128))
    with pytest.raises(TypeError, match="do has dtype"):
        ops.decay_attn_backward(q, k, v, a, do=v.bfloat16())
    with pytest.raises(ValueError, match="act"):
        ops.group_norm(q, act="relu")
    with pytest.raises(ValueError, match="groups"):
        ops.group_norm(c(1, 5, 64), groups=3)
    with pytest.raises(ValueError, match="groups"):
        ops.group_norm(c(1, 5, 64))
    with pytest.raises(ValueError, match="gate"):
        ops.group_norm(q, gate=c(1, 5, 64))
    with pytest.raises(ValueError, match="dy"):
        ops.group_norm_backward(q, c(1, 5, 64))
    with pytest.raises(ValueError, match="no gradients"):
        ops.clip_grad_norm([], 1.0)
    with pytest.raises(ValueError, match="written twice"):
        ops.clip_grad_norm([q, q], 1.0)
    with pytest.raises(ValueError, match="outputs"):
        ops.clip_grad_norm([q, k], 1.0, outs=[v])
    with pytest.raises(ValueError, match="contiguous"):
        ops.clip_grad_norm([c(4, 6).t()], 1.0)
