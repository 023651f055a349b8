"""Gates so far out that their factors leave fp32's normal range (a sigmoid below 2^-126
is one of 87.3), against the formulas in 64 bits.

Tolerance.  A factor is within 3e-5 of itself (an exponential whose argument, up to 151,
rounds by 2^-18), or, below the normal range, within fp32's smallest step, 2^-149, of it;
sqrt(1 - a^2) is taken from e^(-g / 2) there and stays normal to a gate of 174.
"""
import pytest
import torch

from preconditioned_delta_rule_phase1_gb300 import build as osdn_build
from preconditioned_delta_rule_phase1_gb300 import ops

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
REL, STEP = 3e-5, 2.0 ** -149
TINY = {"f32": 2.0 ** -150, "bf16": 2.0 ** -134}   # half a step of the I/O type below its normal range


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    osdn_build.build()
    ops.lib()


def factors64(gate, mix):
    """a, w, a (1 - a) and minus w's derivative."""
    a, b = torch.sigmoid(gate), torch.sigmoid(-gate)
    if mix == "sum":
        return a, torch.ones_like(a), a * b, torch.zeros_like(a)
    if mix == "mean":
        return a, b, a * b, a * b
    return a, (b * (1 + a)).sqrt(), a * b, a * a * (b / (1 + a)).sqrt()


def inputs(io, mix, sign, T):
    """Inputs whose weighted size is about one where fp32 can hold them."""
    gate = sign * torch.cat([torch.arange(80, 128, 0.5), torch.arange(128, 216)])
    C = gate.numel()
    g = torch.Generator().manual_seed(T)
    w = factors64(gate.double(), mix)[1]
    x = (1 + torch.rand(1, T, C, generator=g)).double() * (1 / w).clamp(max=1e38)
    r = (1 + torch.rand(1, C, generator=g)).cuda()
    return gate.expand(1, T, C).contiguous().to(DT[io]).cuda(), x.to(DT[io]).cuda(), r


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("mix", ["sum", "mean", "unit"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("T", [1, 5, 40])
def test_far_gates(io, mix, sign, T):
    gate, x, h0 = inputs(io, mix, sign, T)
    a, w, ab, slope = factors64(gate.double(), mix)
    xd, s = x.double(), h0.double()
    before, states, held = [], [], h0.double().abs()
    size = s.abs()
    for t in range(T):
        before.append(s)
        s = a[:, t] * s + w[:, t] * xd[:, t]
        size = size + (w[:, t] * xd[:, t]).abs()
        states.append(s)
    before, states = torch.stack(before, 1), torch.stack(states, 1)
    if sign < 0:   # (a of 1e-35 and less: what is left of the state before)
        size = torch.maximum(size, before.abs().amax(1))
    tol = REL * size + T * STEP * xd.abs().amax(1)
    h, hT = ops.gated_scan(x, gate, h0, mix=mix)
    off = (h.double() - states).abs() - (HALF[io] * states.abs() + tol[:, None])
    assert bool((off <= 0).all()), gate[0, 0, int(off.amax((0, 1)).argmax())]
    assert bool(((hT.double() - states[:, -1]).abs() <= tol).all())
    state = h0.clone()
    for t in range(T):
        ops.gated_scan_step(x[:, t].clone(), gate[:, t].clone(), state, mix=mix)
    assert bool(((state.double() - states[:, -1]).abs() <= tol).all())
    # gradients, with every R about one (all gates open) or from each token alone (all shut)
    for scale in (1.0, 1e30):
        dh = torch.full_like(x, scale)
        dhT = h0 * scale
        got = ops.gated_scan_backward(x, gate, h, h0, dh=dh, dhT=dhT, mix=mix)
        R, r = torch.empty_like(xd), dhT.double()
        for t in range(T - 1, -1, -1):
            R[:, t] = r = r + dh[:, t].double()
            r = a[:, t] * r
        # (an A or R of shut gates: what fp32 leaves of it)
        dx = w * R
        off = (got["x"].double() - dx).abs() - ((HALF[io] + REL) * dx.abs() + STEP * R + TINY[io])
        assert bool((off <= 0).all()), ("dx", scale, gate[0, 0, int(off.amax((0, 1)).argmax())])
        dg = R * (ab * before - slope * xd)
        terms = REL * R * (ab * before.abs() + slope * xd.abs()) + STEP * R * (before.abs() + xd.abs())
        if T > 1:   # the states are recomputed from rows of h, rounded (of short sequences every fourth)
            terms = terms + R * ab * HALF[io] * states.abs().amax(1, keepdim=True)
        off = (got["gate"].double() - dg).abs() - (HALF[io] * dg.abs() + terms + TINY[io])
        assert bool((off <= 0).all()), ("dgate", scale, gate[0, 0, int(off.amax((0, 1)).argmax())])
        assert bool(((got["h0"].double() - r).abs() <= REL * r + STEP * R[:, 0]).all())


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("mix", ["mean", "unit"])
def test_what_a_finite_gate_does_not_hide(io, mix):
    """A weight that fp32 can say is no zero: an infinite x behind it is read."""
    gate = torch.tensor([[[88.0, 95.0, 100.0, 102.0]]], device="cuda").to(DT[io])
    x = torch.full((1, 1, 4), float("inf"), device="cuda").to(DT[io])
    h0 = torch.zeros(1, 4, device="cuda")
    assert bool((ops.gated_scan(x, gate, h0, mix=mix)[1] == float("inf")).all())
    ops.gated_scan_step(x[:, 0].clone(), gate[:, 0].clone(), h0, mix=mix)
    assert bool((h0 == float("inf")).all())


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_a_far_gate_leaves_its_neighbours_as_they_are(io):
    """A weighted mean of what the state is already does not move: dgate is zero, exactly, whatever form of
    the arithmetic another channel's gate asks for."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(1, 1, 64, generator=g).to(DT[io]).cuda()
    gate = torch.randn(1, 1, 64, generator=g).to(DT[io]).cuda()
    h0 = x[:, 0].float()
    for far in (0.0, float("inf"), 90.0, 150.0, -95.0):
        gate[0, 0, 7] = far
        h, _ = ops.gated_scan(x, gate, h0, mix="mean")
        got = ops.gated_scan_backward(x, gate, h, h0, dh=torch.ones_like(x), mix="mean")
        assert not got["gate"].any(), far
