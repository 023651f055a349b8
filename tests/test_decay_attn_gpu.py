"""Linear attention with a decay per head (osdn_decay_attn, its single-token
step and its gradients) against the token recurrence in 64 bits.

Tolerances, normwise (max |x - ref| / max |ref|).  fp32 I/O sums a few hundred
products in fp32: 2e-5.  bf16 I/O rounds its outputs (2^-9 of their size) and
the operands of the tensor-core products (each term by up to 2^-9, signs
mixed): 1e-2.  The fp32 states see no such rounding in either: 2e-5.
"""
import itertools

import pytest
import torch

from preconditioned_delta_rule_phase1_gb300 import build as osdn_build
from preconditioned_delta_rule_phase1_gb300 import ops
from tests._util import rel_err

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
TOL = {"f32": 2e-5, "bf16": 1e-2}
STATE_TOL = 2e-5
WIDTHS = [(64, 64), (128, 128), (128, 64), (64, 128)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    osdn_build.build()
    ops.lib()


def recurrence(q, k, v, decay, S0=None):
    """The definition, token by token, in 64 bits on the tensors' device."""
    q, k, v, a = (x.double() for x in (q, k, v, decay))
    B, H, T, K = k.shape
    S = torch.zeros(B, H, v.shape[-1], K, dtype=torch.float64, device=k.device) if S0 is None else S0.double()
    o = []
    for t in range(T):
        S = a[:, None, None] * S + v[:, :, t, :, None] * k[:, :, t, None, :]
        o.append(torch.einsum("bhvk,bhk->bhv", S, q[:, :, t]))
    return torch.stack(o, 2), S


def inputs(B, H, T, K, V, io, seed, s0=True, decay=None):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    x = {"q": unit(n(B, H, T, K)).to(DT[io]), "k": unit(n(B, H, T, K)).to(DT[io]),
         "v": n(B, H, T, V).to(DT[io])}
    if decay is None:   # from no memory to all of it
        decay = torch.tensor([0.97, 0.0, 1.0, 0.9995, 1e-3, 0.5, 0.05])[torch.arange(H) % 7]
    x["decay"] = decay
    x["S0"] = n(B, H, V, K) if s0 else None
    x["do"] = n(B, H, T, V).to(DT[io])
    x["dST"] = n(B, H, V, K) if s0 else None
    return {a: None if t is None else t.cuda() for a, t in x.items()}


def forward(x, ws=None):
    return ops.decay_attn(x["q"], x["k"], x["v"], x["decay"], x["S0"], workspace=ws)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("K,V", WIDTHS)
def test_lengths_match_the_recurrence(io, K, V):
    ws = ops.Workspace()
    for T, s0 in itertools.product([1, 2, 15, 63, 64, 65, 127, 128, 129, 200, 257, 385], [False, True]):
        x = inputs(2, 7, T, K, V, io, seed=T + K, s0=s0)
        o, ST = forward(x, ws)
        assert ws.status() == 0
        ro, rS = recurrence(x["q"], x["k"], x["v"], x["decay"], x["S0"])
        assert rel_err(o, ro.cpu()) < TOL[io], T
        assert rel_err(ST, rS.cpu()) < STATE_TOL, T


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,T,K,V", [(1, 1, 3001, 128, 128), (1, 5, 2050, 64, 128), (3, 16, 1111, 128, 64),
                                       (40, 16, 130, 64, 64), (160, 1, 300, 128, 128), (1, 3, 8200, 64, 64)])
def test_every_way_of_cutting_the_time_axis(io, B, H, T, K, V):
    # few long sequences (many ranges each), ranges over several short ones, one a sequence
    x = inputs(B, H, T, K, V, io, seed=T, decay=1.0 - torch.exp2(-torch.linspace(2, 12, H)))
    ws = ops.Workspace()
    o, ST = forward(x, ws)
    assert ws.status() == 0
    ro, rS = recurrence(x["q"], x["k"], x["v"], x["decay"], x["S0"])
    assert rel_err(o, ro.cpu()) < TOL[io]
    assert rel_err(ST, rS.cpu()) < STATE_TOL
    # each head by itself: the decays differ by a factor of a thousand in memory
    for h in range(0, H, 5):
        assert rel_err(ST[:, h], rS[:, h].cpu()) < STATE_TOL
    o2, ST2 = forward(x, ws)
    assert torch.equal(o, o2) and torch.equal(ST, ST2)


def blocks64(q, k, v, decay, S, block=200):
    """The recurrence in 64 bits, block by block (long sequences; autograd passes through)."""
    q, k, v, a = (x.double() for x in (q, k, v, decay))
    S, out = S.double(), []
    for t in range(0, q.shape[2], block):
        qb, kb, vb = (x[:, :, t:t + block] for x in (q, k, v))
        i = torch.arange(qb.shape[2], device=q.device, dtype=torch.float64)
        gap = i[:, None] - i[None, :]
        w = torch.where(gap >= 0, a[:, None, None] ** gap.clamp(min=0), 0.0)
        out.append(((qb @ kb.transpose(-1, -2)) * w) @ vb
                   + (qb @ S.transpose(-1, -2)) * (a[:, None] ** (i + 1))[None, :, :, None])
        S = S * (a ** len(i))[None, :, None, None] + (vb * (a[:, None] ** (len(i) - 1 - i))[None, :, :, None]).transpose(-1, -2) @ kb
    return torch.cat(out, 2), S


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,T,K,V", [(1, 8, 20001, 128, 128), (2, 3, 33000, 64, 64), (1, 16, 30000, 128, 64),
                                       (1, 16, 30000, 64, 128)])
def test_long_ranges(io, B, H, T, K, V):
    # ranges of many units each, forwards and backwards; the states' tolerance is that of fp32
    # sums over a memory of thousands of tokens
    x = inputs(B, H, T, K, V, io, seed=T + K, decay=1.0 - torch.exp2(-torch.linspace(4, 12, H)))
    ws = ops.Workspace()
    o, ST = forward(x, ws)
    got = backward(x, ws)
    assert ws.status() == 0
    t = {n: x[n].double().requires_grad_() for n in ("q", "k", "v", "S0")}
    ro, rS = blocks64(t["q"], t["k"], t["v"], x["decay"], t["S0"])
    assert rel_err(o, ro.detach().cpu()) < TOL[io] and rel_err(ST, rS.detach().cpu()) < STATE_TOL
    # in the mean the state loses nothing against fp32 sums either
    assert float((ST.double() - rS.detach()).norm() / rS.detach().norm()) < 1e-6
    loss = (ro * x["do"].double()).sum() + (rS * x["dST"].double()).sum()
    for n, r in zip(t, torch.autograd.grad(loss, list(t.values()))):
        assert rel_err(got[n], r.cpu()) < (STATE_TOL if n == "S0" else TOL[io]), n
    assert float((got["S0"].double() - r).norm() / r.norm()) < 1e-6


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_prompt_pieces_and_steps_chain(io):
    x = inputs(2, 3, 300, 128, 64, io, seed=5)
    whole, ST = forward(x)
    S, got = x["S0"], []
    for lo, hi in ((0, 1), (1, 140), (140, 297)):
        part = {n: x[n][:, :, lo:hi].contiguous() for n in "qkv"}
        o, S = ops.decay_attn(part["q"], part["k"], part["v"], x["decay"], S)
        got.append(o)
    for t in range(297, 300):   # the last tokens one by one, in place
        got.append(ops.decay_attn_step(*(x[n][:, :, t].contiguous() for n in "qkv"), x["decay"], S)[:, :, None])
    assert rel_err(torch.cat(got, 2), whole.double().cpu()) < 2 * TOL[io]
    assert rel_err(S, ST.double().cpu()) < 2 * STATE_TOL


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("K,V", WIDTHS)
@pytest.mark.parametrize("B,H", [(1, 1), (3, 7), (33, 16)])
def test_step_matches_the_recurrence(io, K, V, B, H):
    x = inputs(B, H, 1, K, V, io, seed=B + K)
    ro, rS = recurrence(x["q"], x["k"], x["v"], x["decay"], x["S0"])
    S = x["S0"].clone()
    ws = ops.Workspace()
    o = ops.decay_attn_step(*(x[n][:, :, 0].contiguous() for n in "qkv"), x["decay"], S, workspace=ws)
    assert ws.status() == 0
    # one product each of the state's terms; o rounds once
    assert rel_err(o, ro[:, :, 0].cpu()) < (2e-5 if io == "f32" else 4e-3)
    assert rel_err(S, rS.cpu()) < 1e-6


def autograd(x):
    t = {n: x[n].double().requires_grad_() for n in "qkv"}
    S0 = x["S0"] if x["S0"] is not None else torch.zeros(x["q"].shape[0], x["q"].shape[1], x["v"].shape[-1],
                                                         x["q"].shape[-1], device="cuda")
    t["S0"] = S0.double().requires_grad_()
    o, ST = recurrence(t["q"], t["k"], t["v"], x["decay"], t["S0"])
    loss = (o * x["do"].double()).sum() + (0 if x["dST"] is None else (ST * x["dST"].double()).sum())
    return dict(zip(t, torch.autograd.grad(loss, list(t.values()))))


def backward(x, ws=None):
    return ops.decay_attn_backward(x["q"], x["k"], x["v"], x["decay"], x["S0"], do=x["do"], dST=x["dST"],
                                   workspace=ws)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("K,V", WIDTHS)
def test_gradients_match_the_formula(io, K, V):
    ws = ops.Workspace()
    for (B, H, T), s0 in itertools.product([(2, 7, 1), (1, 7, 64), (2, 3, 129), (1, 2, 1030), (20, 8, 70)],
                                           [False, True]):
        x = inputs(B, H, T, K, V, io, seed=T + V, s0=s0)
        got, ref = backward(x, ws), autograd(x)
        assert ws.status() == 0
        assert ("S0" in got) == s0
        for n, g in got.items():
            assert rel_err(g, ref[n].cpu()) < (STATE_TOL if n == "S0" else TOL[io]), (n, B, H, T)


def test_gradients_match_differences():
    # the outputs are linear in each of q, k, v and S0, so half the difference of two
    # forward passes along a direction is the derivative but for fp32 rounding
    x = inputs(2, 3, 200, 64, 128, "f32", seed=9, decay=torch.tensor([0.9, 0.999, 1.0]))
    got = backward(x)
    g = torch.Generator(device="cuda").manual_seed(4)
    for n in ("q", "k", "v", "S0"):
        u = torch.randn(x[n].shape, generator=g, device="cuda")
        f = []
        for s in (1.0, -1.0):
            o, ST = forward({**x, n: x[n] + s * u})
            f.append((o.double() * x["do"].double()).sum() + (ST.double() * x["dST"].double()).sum())
        want, have = float(f[0] - f[1]) / 2, float((got[n].double() * u.double()).sum())
        # each pass's sum of products carries 2^-24 of their absolute sum or so
        size = sum(abs(float(y)) for y in f) + float((got[n].double() * u.double()).abs().sum())
        assert abs(want - have) < 2e-5 * size, n


def test_backward_repeats_bit_for_bit():
    x = inputs(1, 4, 2500, 128, 128, "bf16", seed=2, decay=torch.tensor([0.99, 0.999, 1.0, 0.9]))
    a, b = backward(x), backward(x)
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_empty_sequences():
    x = inputs(2, 3, 0, 64, 128, "bf16", seed=1)
    o, ST = forward(x)
    assert o.shape == (2, 3, 0, 128) and torch.equal(ST, x["S0"])
    assert torch.equal(backward(x)["S0"], x["dST"])
    x = inputs(2, 3, 0, 64, 128, "f32", seed=1, s0=False)
    assert not forward(x)[1].any()
    x = inputs(0, 3, 5, 64, 128, "bf16", seed=1)
    assert forward(x)[0].shape == (0, 3, 5, 128)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [1.5, -0.1, float("nan")])
def test_a_decay_out_of_range_is_reported(io, bad):
    for call in ("prompt", "step"):
        x = inputs(1, 3, 70 if call == "prompt" else 1, 64, 64, io, seed=3,
                   decay=torch.tensor([0.5, bad, 1.0]))
        ws = ops.Workspace()
        if call == "prompt":
            forward(x, ws)
        else:
            ops.decay_attn_step(*(x[n][:, :, 0].contiguous() for n in "qkv"), x["decay"], x["S0"], workspace=ws)
        assert ws.status() == -8
        ws.reset()
        torch.cuda.synchronize()
        assert ws.status() == 0


def test_on_another_stream_and_in_a_graph():
    x = inputs(1, 4, 700, 128, 128, "bf16", seed=8, decay=torch.tensor([0.99, 0.999, 1.0, 0.9]))
    want, gw = forward(x), backward(x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    ws, wb = ops.Workspace(), ops.Workspace()
    with torch.cuda.stream(side):
        o, ST = forward(x, ws)
        g = backward(x, wb)
    side.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(ST, want[1])
    assert all(torch.equal(g[n], gw[n]) for n in g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.decay_attn(x["q"], x["k"], x["v"], x["decay"], x["S0"], o=o, ST=ST, workspace=ws)
    x["v"].mul_(-1.0)   # every output but S0's share changes sign
    x["S0"].mul_(-1.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, -want[0]) and torch.equal(ST, -want[1])


def test_a_wait_that_runs_out_is_reported():
    # while the workspace's test word is nonzero the bf16 kernel loads nothing and its waits
    # are shortened: they run out, the status says so and the device stays usable
    x = inputs(1, 2, 300, 64, 64, "bf16", seed=3)
    want = forward(x)
    ws = ops.Workspace()
    ws.ensure(ops.decay_attn_workspace_bytes(1, 1, 2, 300, 64, 64))
    ws.buf[4] = 1
    forward(x, ws)
    assert ws.status() == -7
    ws.reset()
    o, ST = forward(x, ws)
    assert ws.status() == 0 and torch.equal(o, want[0]) and torch.equal(ST, want[1])
