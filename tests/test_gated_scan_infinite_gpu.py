"""Infinite states and cotangents through osdn_gated_scan, its step and its gradients:
a v is an infinity where v is one and a is not zero, and stays hidden where a is zero.

The reference is the definition in 64 bits, in which a factor of zero hides what it
multiplies.  Where it is an infinity or NaN the result has to be the same one; the rest
is as close as in the other tests of these calls: half a step of the I/O type (below the
normal range: half of the type's smallest step, 2^-134 in bf16) and 3e-5 of the channel's
largest finite value.  The last state's channel is what its tokens' states are, too: a
state near zero is a sum of terms as large as those, and their roundings stay.
"""
import math

import pytest
import torch

from preconditioned_delta_rule_phase1_gb300 import build as osdn_build
from preconditioned_delta_rule_phase1_gb300 import ops

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
TOL32 = 3e-5
MIXES = ["sum", "mean", "unit"]
INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    osdn_build.build()
    ops.lib()


def hide(c, v):
    return torch.where(c == 0, torch.zeros_like(v), c * v)


def gates64(gate, mix):
    """a, 1 - a, w and the k of w' = -a (1 - a) k."""
    a, b = torch.sigmoid(gate), torch.sigmoid(-gate)
    if mix == "sum":
        return a, b, torch.ones_like(a), torch.zeros_like(a)
    if mix == "mean":
        return a, b, b, torch.ones_like(a)
    return a, b, (b * (1 + a)).sqrt(), a / (b * (1 + a)).sqrt()


def forward64(x, gate, h0, mix):
    a, _, w, _ = gates64(gate, mix)
    wx, s, before, out = hide(w, x), h0, [], []
    for t in range(x.shape[1]):
        before.append(s)
        s = hide(a[:, t], s) + wx[:, t]
        out.append(s)
    return torch.stack(out, 1), torch.stack(before, 1)


def backward64(x, gate, h0, mix, dh, dhT, half):
    a, b, w, k = gates64(gate, mix)
    _, before = forward64(x, gate, h0, mix)
    R, r = torch.empty_like(x), dhT
    for t in range(x.shape[1] - 1, -1, -1):
        R[:, t] = r = r + dh[:, t]
        r = hide(a[:, t], r)
    ab = a * b
    slope = hide(ab, before) - hide(torch.where(ab == 0, ab, ab * k), x)
    # where the slope's sign is known although the states it is made of were rounded to be stored
    held = torch.where(torch.isfinite(before), before, torch.zeros_like(before)).abs().amax(1, keepdim=True)
    sure = slope.abs() > ab * held * (half + TOL32)
    return hide(w, R), torch.where(ab == 0, torch.zeros_like(R), R * slope), r, sure


def same(got, ref, half, what, among=None):
    got = got.double()
    bad = ~torch.isfinite(ref)
    assert torch.equal(torch.isfinite(got), ~bad), what
    assert torch.equal(got.isnan(), ref.isnan()) and torch.equal(got == INF, ref == INF), what
    ref, got = ref.masked_fill(bad, 0), got.masked_fill(bad, 0)
    among = ref if among is None else among.masked_fill(~torch.isfinite(among), 0)
    size = among.abs().amax(tuple(range(among.dim() - 1)))
    off = (got - ref).abs() - (half * ref.abs() + TOL32 * size + 2.0 ** -134)
    assert bool((off <= 0).all()), (what, float(off.max()))


def gates(B, T, C, io, kind):
    """kind: a number for a constant gate, "mixed" for moderate ones, "pass" for moderate ones of which
    some are +inf."""
    g = torch.Generator().manual_seed(T)
    gate = torch.randn(B, T, C, generator=g) * 2 + 1
    if kind == "pass":
        gate = torch.where(torch.rand(B, T, C, generator=g) < 0.3, INF, gate)
    elif kind != "mixed":
        gate = torch.full((B, T, C), float(kind))
    return gate.to(DT[io]).cuda()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("mix", MIXES)
@pytest.mark.parametrize("kind", [INF, 2.0, -2.0, 0.0, 50.0, 84.0, -85.0, "mixed", "pass"])
def test_an_infinite_state_stays_infinite(io, mix, kind):
    """From h0 and from x, at lengths that end inside a warp's tokens, and at whole ones."""
    for T, C in ((1, 5), (3, 64), (130, 33), (256, 64), (1025, 20), (2048, 6)):
        g = torch.Generator().manual_seed(T + 1)
        x, h0 = torch.randn(2, T, C, generator=g), torch.randn(2, C, generator=g)
        h0[0, 0], h0[0, 1], h0[1, 2] = INF, -INF, math.nan
        x[1, T // 2, 3], x[1, T - 1, 4], x[0, T // 3, 4] = -INF, INF, INF
        x, h0, gate = x.to(DT[io]).cuda(), h0.cuda(), gates(2, T, C, io, kind)
        ref, _ = forward64(x.double(), gate.double(), h0.double(), mix)
        if kind == -85.0:
            # a is 1e-37: the gates' product leaves fp32 within two tokens, and what it multiplies with it
            ref, T = ref[:, :1], 1
            x, gate = x[:, :1].contiguous(), gate[:, :1].contiguous()
        h, hT = ops.gated_scan(x, gate, h0, mix=mix)
        if kind in ("mixed", 2.0, -2.0, 0.0) and T > 15:
            # the same for moderate gates some tokens on: an infinity lives as long as their product does
            a = torch.sigmoid(gate.double()).log().cumsum(1)
            assert float(a[:, 15].min()) > math.log(2.0 ** -126)
            ref, h = ref[:, :15], h[:, :15]
            same(h, ref, HALF[io], (T, C, "h"))
            continue
        same(h, ref, HALF[io], (T, C, "h"))
        same(hT, ref[:, -1], 2.0 ** -24, (T, C, "hT"), among=ref)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("mix", MIXES)
@pytest.mark.parametrize("kind", [INF, 2.0, -2.0, 0.0, 84.0, "mixed", "pass"])
def test_a_step_keeps_an_infinite_state(io, mix, kind):
    g = torch.Generator().manual_seed(7)
    x, gate = torch.randn(3, 1, 37, generator=g).to(DT[io]).cuda(), gates(3, 1, 37, io, kind)
    h0 = torch.randn(3, 37, generator=g).cuda()
    h0[0, ::2], h0[1, 1::2], h0[2, 5] = INF, -INF, math.nan
    x[2, 0, 7] = INF
    ref, _ = forward64(x.double(), gate.double(), h0.double(), mix)
    state = h0.clone()
    y = ops.gated_scan_step(x[:, 0].contiguous(), gate[:, 0].contiguous(), state, mix=mix)
    terms = torch.cat([h0.double(), x[:, 0].double(), ref[:, 0]])   # the sum is rounded as its two terms are
    same(y, ref[:, 0], HALF[io], "y", among=terms)
    same(state, ref[:, 0], 2.0 ** -24, "h", among=terms)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("mix", MIXES)
@pytest.mark.parametrize("kind", [INF, 2.0, 50.0, 84.0, "mixed", "pass"])
@pytest.mark.parametrize("T", [1, 5, 15, 300, 1025])
def test_infinite_cotangents_and_states_backwards(io, mix, kind, T):
    """An infinite dhT reaches the tokens before it as an infinity, an infinite h0 the dgate of its channel."""
    if T > 15 and kind in (2.0, "mixed"):
        T = 15   # (as above)
    C = 34
    g = torch.Generator().manual_seed(T)
    x, dh = (torch.randn(2, T, C, generator=g).to(DT[io]).cuda() for _ in range(2))
    h0, dhT = (torch.randn(2, C, generator=g).cuda() for _ in range(2))
    gate = gates(2, T, C, io, kind)
    h0[0, 0], h0[1, 1], dhT[0, 2], dhT[1, 3], dhT[1, 33] = INF, -INF, INF, -INF, math.nan
    dh[1, T // 2, 4] = INF
    h, _ = ops.gated_scan(x, gate, h0, mix=mix)
    got = ops.gated_scan_backward(x, gate, h, h0, dh=dh, dhT=dhT, mix=mix)
    dx, dg, dh0, sure = backward64(x.double(), gate.double(), h0.double(), mix, dh.double(), dhT.double(), HALF[io])
    same(got["x"], dx, HALF[io], "dx")
    same(got["h0"], dh0, 2.0 ** -24, "dh0")
    bad = ~torch.isfinite(dg)
    assert torch.equal(~torch.isfinite(got["gate"]), bad)
    sure |= dg.isnan()
    assert torch.equal((got["gate"].double() == INF)[sure], (dg == INF)[sure])
    assert torch.equal(got["gate"].isnan()[sure], dg.isnan()[sure])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("mix", MIXES)
@pytest.mark.parametrize("T", [1, 6, 300, 2000])
def test_a_gate_of_nan_reaches_its_channel_until_a_restart(io, mix, T):
    C, at = 34, T // 3
    g = torch.Generator().manual_seed(T)
    x, dh = (torch.randn(2, T, C, generator=g).to(DT[io]).cuda() for _ in range(2))
    h0, dhT = (torch.randn(2, C, generator=g).cuda() for _ in range(2))
    gate = gates(2, T, C, io, "mixed")
    gate[1, at, 5] = math.nan
    if T > 5:
        gate[:, at + 3] = -INF
    ref, _ = forward64(x.double(), gate.double(), h0.double(), mix)
    h, hT = ops.gated_scan(x, gate, h0, mix=mix)
    assert torch.equal(h.isnan(), ref.isnan()) and int(h.isnan().sum()) == min(3, T - at)
    same(h, ref, HALF[io], "h")
    same(hT, ref[:, -1], 2.0 ** -24, "hT", among=ref)
    got = ops.gated_scan_backward(x, gate, h, h0, dh=dh, dhT=dhT, mix=mix)
    # R of the tokens before is NaN, w and the slope of the token itself are, and the slopes behind it
    w = torch.ones(T, dtype=torch.bool, device="cuda")
    before, after = w.clone(), w.clone()
    before[at:], after[:at + 1], after[at + 3:] = False, False, False   # (the restart's own slope is zero)
    want = torch.zeros(2, T, C, dtype=torch.bool, device="cuda")
    want[1, :, 5] = before
    if mix != "sum":
        want[1, at, 5] = True
    assert torch.equal(got["x"].isnan(), want)
    want[1, at, 5] = True
    want[1, :, 5] |= after
    assert torch.equal(got["gate"].isnan(), want)
    assert int(got["h0"].isnan().sum()) == 1 and bool(got["h0"][1, 5].isnan())


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("mix", MIXES)
@pytest.mark.parametrize("T,C,B", [(1, 33, 3), (4, 5, 180), (6, 33, 5), (16, 64, 4), (40, 130, 2), (100, 34, 3), (700, 20, 2)])
def test_infinities_nan_and_restarts_together(io, mix, T, C, B):
    """Gates of +-inf, NaN and 90 and infinite or NaN values, all over a call: the same ones come out, at the
    same places.  (The gates between are open enough for their product to stay in fp32.)"""
    for seed in range(4):
        g = torch.Generator().manual_seed(seed * 1000 + T)
        some = lambda p, *s: torch.rand(*s, generator=g) < p  # noqa: E731
        gate = (1 if T < 200 else 4) + 4 * torch.rand(B, T, C, generator=g)
        gate = torch.where(some(0.04, B, T, 1), -INF, gate)
        if seed % 2:
            gate = torch.where(some(0.1, B, T, 1), INF, gate)
        gate = torch.where(some(0.01, B, T, C), math.nan, gate)
        gate = torch.where(some(0.02, B, T, C), 90.0, gate)
        x, dh = (torch.randn(B, T, C, generator=g) for _ in range(2))
        h0, dhT = (torch.randn(B, C, generator=g) for _ in range(2))
        for i, t in enumerate((x, dh, h0, dhT)):
            for k, v in enumerate((INF, -INF, math.nan)):
                if (seed + i + k) % 3 == 0:
                    t[some(0.03, *t.shape)] = v
        x, dh, gate, h0, dhT = x.to(DT[io]).cuda(), dh.to(DT[io]).cuda(), gate.to(DT[io]).cuda(), h0.cuda(), dhT.cuda()
        ref, _ = forward64(x.double(), gate.double(), h0.double(), mix)
        h, hT = ops.gated_scan(x, gate, h0, mix=mix)
        same(h, ref, HALF[io], ("h", seed))
        same(hT, ref[:, -1], 2.0 ** -24, ("hT", seed), among=ref)
        got = ops.gated_scan_backward(x, gate, h, h0, dh=dh, dhT=dhT, mix=mix)
        dx, dg, dh0, sure = backward64(x.double(), gate.double(), h0.double(), mix, dh.double(), dhT.double(), HALF[io])
        for name, a, b in (("x", got["x"], dx), ("h0", got["h0"], dh0)):
            assert torch.equal(a.isnan(), b.isnan()), (name, seed)
            assert torch.equal(a.double() == INF, b == INF) and torch.equal(a.double() == -INF, b == -INF), (name, seed)
        sure |= dg.isnan()
        assert torch.equal(torch.isfinite(got["gate"])[sure], torch.isfinite(dg)[sure]), seed
        assert torch.equal((got["gate"].double() == INF)[sure], (dg == INF)[sure]), seed
