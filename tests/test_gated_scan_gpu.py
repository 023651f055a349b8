"""The gated recurrence (osdn_gated_scan, its step and its gradients) against the
token recurrence in 64 bits.

Tolerances.  An I/O rounding is off by at most half a step of the value itself
(bf16 2^-8, fp32 2^-24).  The arithmetic is fp32: a gate is within about 2^-21
(an exponential, a quotient and a root of a few ulp each), and a state is a sum
over its memory, 1 / (1 - a) tokens, each of which rounds twice; with memories up
to 4000 tokens the roundings, as a random walk, are within 8 sqrt(4000) 2^-24 =
3e-5 of the largest value of the channel.  TOL32 is that.  A gradient of the gate
reads a state that is recomputed from a stored row of h, off by half a step of
that row at most (and less with every token behind it), and by the arithmetic behind that row.
"""
import itertools
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


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    osdn_build.build()
    ops.lib()


def gates64(gate, mix):
    """a, 1 - a, w and w's derivative by the gate."""
    a, b = torch.sigmoid(gate), torch.sigmoid(-gate)
    if mix == "sum":
        return a, b, torch.ones_like(a), torch.zeros_like(a)
    if mix == "mean":
        return a, b, b, -a * b
    return a, b, (b * (1 + a)).sqrt(), -a * a * (b / (1 + a)).sqrt()


def hide(c, v):
    return torch.where(c == 0, torch.zeros_like(v), c * v)


def forward64(x, gate, h0, mix):
    """All states [B,T,C] and the one before each."""
    a, b, w, _ = gates64(gate, mix)
    wx = hide(w, x)
    s = torch.zeros_like(x[:, 0]) if h0 is None else h0
    before, out = [], []
    for t in range(x.shape[1]):
        before.append(s)
        s = hide(a[:, t], s) + wx[:, t]
        out.append(s)
    return torch.stack(out, 1), torch.stack(before, 1)


def backward64(x, gate, h0, mix, dh, dhT):
    """dx, dgate, dh0, and |R| a (1 - a): what an error of the state is multiplied with."""
    a, b, w, slope = gates64(gate, mix)
    _, before = forward64(x, gate, h0, mix)
    R = torch.empty_like(x)
    r = torch.zeros_like(x[:, 0]) if dhT is None else dhT
    for t in range(x.shape[1] - 1, -1, -1):
        R[:, t] = r = r + dh[:, t]
        r = hide(a[:, t], r)
    return w * R, R * (hide(a * b, before) + hide(slope, x)), r, R.abs() * a * b


def inputs(B, T, C, io, seed, h0=True, low=-2.0, high=8.0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    gate = low + (high - low) * torch.rand(C, generator=g) + n(B, T, C)
    return {"x": n(B, T, C).to(DT[io]).cuda(), "gate": gate.to(DT[io]).cuda(),
            "h0": n(B, C).cuda() if h0 else None, "dh": n(B, T, C).to(DT[io]).cuda(),
            "dhT": n(B, C).cuda() if h0 else None}


def wide(t):
    return {k: None if v is None else v.double() for k, v in t.items()}


def close(got, ref, half, extra=0.0, what=""):
    """Every element within half a step of its own size and TOL32 of its channel's largest."""
    assert got.shape == ref.shape, what
    if not ref.numel():
        return
    size = ref.abs().amax(tuple(range(ref.dim() - 1)))
    off = (got.double() - ref).abs() - (half * ref.abs() + TOL32 * size + extra)
    assert bool((off <= 0).all()), (what, float(off.max()), float(size.max()))


def check(t, mix, io, ws, what=""):
    d = wide(t)
    ref, _ = forward64(d["x"], d["gate"], d["h0"], mix)
    h, hT = ops.gated_scan(t["x"], t["gate"], t["h0"], mix=mix, workspace=ws)
    close(h, ref, HALF[io], what=("h", what))
    close(hT, ref[:, -1], 2.0 ** -24, TOL32 * ref.abs().amax((0, 1)), what=("hT", what))
    dx, dg, dh0, lever = backward64(d["x"], d["gate"], d["h0"], mix, d["dh"], d["dhT"])
    got = ops.gated_scan_backward(t["x"], t["gate"], h, t["h0"], dh=t["dh"], dhT=t["dhT"], mix=mix, workspace=ws)
    assert sorted(got) == sorted(["x", "gate"] + (["h0"] if t["h0"] is not None else []))
    close(got["x"], dx, HALF[io], what=("dx", what))
    close(got["gate"], dg, HALF[io], lever * ((HALF[io] + TOL32) * ref.abs().amax((0, 1))), what=("dgate", what))
    if t["h0"] is not None:
        R = dx / gates64(d["gate"], mix)[2]
        close(got["h0"], dh0, 2.0 ** -24, TOL32 * torch.nan_to_num(R.abs(), 0.0, 0.0, 0.0).amax((0, 1)),
              what=("dh0", what))


LENGTHS = [1, 2, 3, 7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 511, 513, 700]
WIDTHS = [1, 2, 3, 31, 32, 33, 62, 64, 65, 66, 100, 128, 130]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("mix", MIXES)
def test_lengths(io, mix):
    ws = ops.Workspace()
    for i, T in enumerate(LENGTHS):
        for C in (WIDTHS[i % len(WIDTHS)], WIDTHS[(i + 5) % len(WIDTHS)]):
            check(inputs(1 + i % 3, T, C, io, seed=i, h0=bool(i % 2)), mix, io, ws, (T, C))
    assert ws.status() == 0


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("T,C,B", [(1023, 64, 1), (1024, 62, 2), (1025, 33, 1), (2047, 64, 1), (2049, 130, 2),
                                   (4096, 64, 1), (4097, 20, 3), (9000, 66, 1), (1500, 690, 1), (700, 2048, 2)])
def test_long(io, T, C, B):
    ws = ops.Workspace()
    for mix in MIXES:
        check(inputs(B, T, C, io, seed=T, h0=T % 2 == 0), mix, io, ws, (T, C, mix))
    assert ws.status() == 0


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_very_long_narrow_and_short_wide(io):
    ws = ops.Workspace()
    check(inputs(1, 40000, 6, io, seed=1), "mean", io, ws)
    check(inputs(1, 20001, 7, io, seed=2), "unit", io, ws)
    check(inputs(2, 5, 5000, io, seed=3), "sum", io, ws)
    check(inputs(700, 3, 40, io, seed=4), "mean", io, ws)
    assert ws.status() == 0


def test_many_strips():
    """More sequences than a dimension of the grid but the first holds."""
    ws = ops.Workspace()
    check(inputs(70000, 2, 3, "bf16", seed=4), "mean", "bf16", ws)
    assert ws.status() == 0


@pytest.mark.parametrize("mix", MIXES)
@pytest.mark.parametrize("T", [1, 40, 300, 5000])
def test_memories_without_end(mix, T):
    """Gates up to 17 (1 - a = 4e-8, less than fp32 can say of a): the state hardly decays."""
    t = inputs(1, T, 64, "f32", seed=T, low=9.0, high=16.0)
    check(t, mix, "f32", None, T)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("mix", MIXES)
def test_restarts_and_padding(io, mix):
    """A gate of -inf forgets: each document is what it is alone, whatever the ones before hold.
    A gate of +inf passes over a token, whatever it holds (where w is then zero)."""
    ws = ops.Workspace()
    for T, C in ((50, 33), (700, 64), (3000, 40)):
        t = inputs(2, T, C, io, seed=T)
        cut = T // 3
        t["gate"][:, cut] = -math.inf
        t["x"][:, cut - 2] = math.nan
        t["x"][0, cut // 2] = math.inf
        h, hT = ops.gated_scan(t["x"], t["gate"], t["h0"], mix=mix, workspace=ws)
        alone, aT = ops.gated_scan(t["x"][:, cut:].contiguous(), t["gate"][:, cut:].contiguous(), None, mix=mix,
                                   workspace=ws)
        assert h[:, cut - 2:cut].isnan().all() and torch.isfinite(h[:, cut:]).all() and torch.isfinite(hT).all()
        ref, _ = forward64(t["x"][:, cut:].double(), t["gate"][:, cut:].double(), None, mix)
        for got, end in ((h[:, cut:], hT), (alone, aT)):
            close(got, ref, HALF[io])
            close(end, ref[:, -1], 2.0 ** -24, TOL32 * ref.abs().amax((0, 1)))
        # no cotangent reaches the documents before, and NaN in their states none after
        t["dh"][:, :cut] = 0
        g = ops.gated_scan_backward(t["x"], t["gate"], h, t["h0"], dh=t["dh"], dhT=t["dhT"], mix=mix, workspace=ws)
        # (zero cotangents times NaN states are NaN: the rows before the NaN are clean)
        assert not g["x"][:, :cut].any() and not g["gate"][:, :cut // 2].any() and not g["h0"].any()
        assert torch.isfinite(g["gate"][:, cut:]).all() and torch.isfinite(g["x"][:, cut:]).all()
        if mix == "sum":
            continue
        t = inputs(2, T, C, io, seed=T + 1)
        t["gate"][0, T // 2:] = math.inf
        t["x"][0, T // 2:] = math.nan
        t["gate"][1, 5:9] = math.inf
        t["x"][1, 5:9] = -math.inf
        t["dh"][0, T // 2:] = 0
        check_padded(t, mix, io, ws)
    assert ws.status() == 0


def check_padded(t, mix, io, ws):
    d = wide(t)
    ref, _ = forward64(d["x"], d["gate"], d["h0"], mix)
    assert torch.isfinite(ref).all()
    h, hT = ops.gated_scan(t["x"], t["gate"], t["h0"], mix=mix, workspace=ws)
    close(h, ref, HALF[io])
    close(hT, ref[:, -1], 2.0 ** -24, TOL32 * ref.abs().amax((0, 1)))
    T = h.shape[1]
    dx, dg, dh0, lever = backward64(d["x"], d["gate"], d["h0"], mix, d["dh"], d["dhT"])
    g = ops.gated_scan_backward(t["x"], t["gate"], h, t["h0"], dh=t["dh"], dhT=t["dhT"], mix=mix, workspace=ws)
    close(g["x"], dx, HALF[io])
    close(g["gate"], dg, HALF[io], lever * ((HALF[io] + TOL32) * ref.abs().amax((0, 1))))
    assert not g["x"][0, T // 2:].any() and not g["gate"][0, T // 2:].any()


@pytest.mark.parametrize("T", [5, 300, 5000])
def test_extreme_gates(T):
    """Finite gates whose sigmoid leaves fp32, on both sides."""
    t = inputs(1, T, 48, "f32", seed=9)
    t["gate"][:, :, 0::4] = 200.0
    t["gate"][:, :, 1::4] = -200.0
    t["gate"][:, :, 2::4] = torch.where(torch.rand(1, T, 12, device="cuda") < 0.5, 95.0, -95.0)
    for mix in MIXES:
        d = wide(t)
        ref, _ = forward64(d["x"], d["gate"], d["h0"], mix)
        h, hT = ops.gated_scan(t["x"], t["gate"], t["h0"], mix=mix)
        close(h, ref, 2.0 ** -24, what=mix)
        dx, dg, dh0, lever = backward64(d["x"], d["gate"], d["h0"], mix, d["dh"], d["dhT"])
        g = ops.gated_scan_backward(t["x"], t["gate"], h, t["h0"], dh=t["dh"], dhT=t["dhT"], mix=mix)
        assert all(torch.isfinite(v).all() for v in g.values())
        # a sigmoid below fp32's normal range (2^-126) may be zero, and the root of twice it with it
        R = (dx / gates64(d["gate"], mix)[2]).abs() * 2.0 ** (-62 if mix == "unit" else -126)
        close(g["x"], dx, 2.0 ** -24, R, what=mix)
        close(g["gate"], dg, 2.0 ** -24, R * d["x"].abs() + lever * 2.0 ** -126 + 1e-30, what=mix)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("mix", MIXES)
def test_large_and_small_values(io, mix):
    """Nothing on the way leaves fp32 where the results do not: inputs of 1e30 behind gates up to 79 and
    down to -79, and values of 1e-30."""
    for size in (1e30, 1e-30):
        t = inputs(1, 300, 66, io, seed=11)
        t["gate"][:, :, 0::3] = 79.0
        t["gate"][:, :, 1::3] = torch.where(torch.rand(1, 300, 22, device="cuda") < 0.5, 60.0, -79.0).to(DT[io])
        for n in ("x", "h0"):
            t[n] *= size
        d = wide(t)
        ref, _ = forward64(d["x"], d["gate"], d["h0"], mix)
        h, hT = ops.gated_scan(t["x"], t["gate"], t["h0"], mix=mix)
        close(h, ref, HALF[io], 1e-37, what=(mix, size))
        dx, dg, dh0, lever = backward64(d["x"], d["gate"], d["h0"], mix, d["dh"], d["dhT"])
        g = ops.gated_scan_backward(t["x"], t["gate"], h, t["h0"], dh=t["dh"], dhT=t["dhT"], mix=mix)
        assert all(torch.isfinite(v).all() for v in g.values()), (mix, size)
        # (values below fp32's normal range may be zero)
        close(g["x"], dx, HALF[io], 1e-36, what=(mix, size))
        close(g["gate"], dg, HALF[io], lever * ((HALF[io] + TOL32) * ref.abs().amax((0, 1))) + 1e-36, what=(mix, size))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("mix", MIXES)
@pytest.mark.parametrize("B,C", [(1, 1), (1, 2048), (3, 33), (256, 130), (70001, 3)])
def test_steps_follow_the_prompt(io, mix, B, C):
    t = inputs(B, 6, C, io, seed=B)
    d = wide(t)
    ref, _ = forward64(d["x"], d["gate"], d["h0"], mix)
    s = t["h0"].clone()
    for i in range(6):
        y = ops.gated_scan_step(t["x"][:, i].clone(), t["gate"][:, i].clone(), s, mix=mix)
        close(y, ref[:, i], HALF[io], TOL32 * ref.abs().amax((0, 1)))
        close(s, ref[:, i], 2.0 ** -24, TOL32 * ref.abs().amax((0, 1)))
    # a prompt in pieces, read on from a state
    h1, s1 = ops.gated_scan(t["x"][:, :2].clone(), t["gate"][:, :2].clone(), t["h0"], mix=mix)
    h2, s2 = ops.gated_scan(t["x"][:, 2:].clone(), t["gate"][:, 2:].clone(), s1, mix=mix)
    close(torch.cat([h1, h2], 1), ref, HALF[io])
    close(s2, s.double(), 2.0 ** -24, TOL32 * ref.abs().amax((0, 1)))


@pytest.mark.parametrize("mix", MIXES)
@pytest.mark.parametrize("T", [3, 50, 400])
def test_gradients_match_differences(mix, T):
    t = inputs(2, T, 40, "f32", seed=T, low=-1.0, high=4.0)
    h, _ = ops.gated_scan(t["x"], t["gate"], t["h0"], mix=mix)
    got = ops.gated_scan_backward(t["x"], t["gate"], h, t["h0"], dh=t["dh"], dhT=t["dhT"], mix=mix)
    g = torch.Generator(device="cuda").manual_seed(1)
    step = 2.0 ** -8
    args = {n: t[n] for n in ("x", "gate", "h0")}

    def loss(**kw):
        h, hT = ops.gated_scan(**{**args, **kw}, mix=mix)
        return float((h.double() * t["dh"].double()).sum() + (hT.double() * t["dhT"].double()).sum())
    for n in args:
        u = torch.randn(args[n].shape, generator=g, device="cuda")
        want = (loss(**{n: args[n] + step * u}) - loss(**{n: args[n] - step * u})) / (2 * step)
        terms = got[n].double() * u.double()
        # central differences: step^2 (1.5e-5) of third derivatives, each of order 1 to 10 times the
        # first ones, plus fp32 rounding over step; against the root of the sum of squares
        assert abs(want - float(terms.sum())) < 1e-2 * float(terms.square().sum().sqrt()), n


def test_optional_arguments():
    t = inputs(2, 300, 66, "bf16", seed=3)
    d = wide(t)
    h, hT = ops.gated_scan(t["x"], t["gate"], mix="unit")
    ref, _ = forward64(d["x"], d["gate"], None, "unit")
    close(h, ref, HALF["bf16"])
    for h0, dhT in itertools.product([None, t["h0"]], [None, t["dhT"]]):
        h, _ = ops.gated_scan(t["x"], t["gate"], h0, mix="unit")
        ref, _ = forward64(d["x"], d["gate"], None if h0 is None else d["h0"], "unit")
        dx, dg, dh0, lever = backward64(d["x"], d["gate"], None if h0 is None else d["h0"], "unit", d["dh"],
                                        None if dhT is None else d["dhT"])
        g = ops.gated_scan_backward(t["x"], t["gate"], h, h0, dh=t["dh"], dhT=dhT, mix="unit")
        close(g["x"], dx, HALF["bf16"])
        close(g["gate"], dg, HALF["bf16"], lever * ((HALF["bf16"] + TOL32) * ref.abs().amax((0, 1))))
        assert ("h0" in g) == (h0 is not None)
    # given outputs are written, and nothing beside them
    room = torch.full((3, 2, 300, 66), 7.0, dtype=torch.bfloat16, device="cuda")
    end = torch.full((3, 2, 66), 7.0, device="cuda")
    out = ops.gated_scan(t["x"], t["gate"], t["h0"], mix="unit", h=room[1], hT=end[1])
    assert out[0].data_ptr() == room[1].data_ptr() and out[1].data_ptr() == end[1].data_ptr()
    assert bool((room[::2] == 7).all()) and bool((end[::2] == 7).all())
    want = ops.gated_scan(t["x"], t["gate"], t["h0"], mix="unit")
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_empty():
    x = torch.empty(2, 0, 32, device="cuda")
    h0 = torch.randn(2, 32, device="cuda")
    h, hT = ops.gated_scan(x, x, h0)
    assert h.shape == (2, 0, 32) and torch.equal(hT, h0)
    assert not ops.gated_scan(x, x)[1].any()
    g = ops.gated_scan_backward(x, x, h, h0, dh=x, dhT=h0 + 1)
    assert torch.equal(g["h0"], h0 + 1) and g["x"].shape == (2, 0, 32)
    for shape in ((0, 5, 32), (2, 5, 0)):
        e = torch.empty(*shape, device="cuda")
        assert ops.gated_scan(e, e)[0].shape == shape
        assert ops.gated_scan_backward(e, e, e, dh=e)["x"].shape == shape
    e = torch.empty(0, 32, device="cuda")
    assert ops.gated_scan_step(e, e, e).shape == (0, 32)


@pytest.mark.parametrize("T,C", [(300, 66), (1100, 33), (6000, 130)])
def test_repeatable_and_elsewhere(T, C):
    t = inputs(2, T, C, "bf16", seed=6)
    ws = ops.Workspace()

    def run(stream=None):
        h, hT = ops.gated_scan(t["x"], t["gate"], t["h0"], mix="mean", workspace=ws, stream=stream)
        g = ops.gated_scan_backward(t["x"], t["gate"], h, t["h0"], dh=t["dh"], dhT=t["dhT"], mix="mean",
                                    workspace=ws, stream=stream)
        return [h, hT, g["x"], g["gate"], g["h0"]]
    want = run()
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(run(), want))
    ws.buf[256:] = 0x5a   # whatever an earlier call has left
    assert all(torch.equal(a, b) for a, b in zip(run(), want))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = run(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # two calls at once, each with its workspace
    other = ops.Workspace()
    torch.cuda.synchronize()
    pairs = []
    for _ in range(5):
        pairs.append(run())
        with torch.cuda.stream(side):
            h, hT = ops.gated_scan(t["x"], t["gate"], t["h0"], mix="mean", workspace=other)
            g = ops.gated_scan_backward(t["x"], t["gate"], h, t["h0"], dh=t["dh"], dhT=t["dhT"], mix="mean",
                                        workspace=other)
            pairs.append([h, hT, g["x"], g["gate"], g["h0"]])
    torch.cuda.synchronize()
    for p in pairs:
        assert all(torch.equal(a, b) for a, b in zip(p, want))
    assert ws.status() == 0 and other.status() == 0


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("T", [70, 600, 5000])
def test_in_a_graph(io, T):
    t = inputs(2, T, 66, io, seed=4)
    ws, state = ops.Workspace(), torch.zeros(2, 66, device="cuda")
    x1, g1 = t["x"][:, 0].contiguous(), t["gate"][:, 0].contiguous()

    def run(s):
        h, hT = ops.gated_scan(t["x"], t["gate"], t["h0"], mix="unit", workspace=ws)
        g = ops.gated_scan_backward(t["x"], t["gate"], h, t["h0"], dh=t["dh"], dhT=t["dhT"], mix="unit",
                                    workspace=ws)
        return [h, hT, g["x"], g["gate"], g["h0"], ops.gated_scan_step(x1, g1, s, mix="unit")]
    run(state)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(state)
    for i in range(3):
        t["x"].mul_(-1.5)
        t["gate"].add_(0.25)
        state.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = run(torch.zeros(2, 66, device="cuda"))
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
    assert ws.status() == 0


def test_offsets_past_32_bits():
    """More than 2^31 elements a tensor: the last tokens are what they are alone, behind a restart, and
    so are the first ones' gradients."""
    T, C, part = 1100001, 1990, 3000
    assert T * C > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(1)
    x, gate, dh = (torch.empty(1, T, C, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(3))
    gate.add_(3.0)
    gate[:, part] = gate[:, T - part] = -math.inf
    h, hT = ops.gated_scan(x, gate, mix="mean")
    tail = slice(T - part, T)
    alone, aT = ops.gated_scan(x[:, tail].clone(), gate[:, tail].clone(), mix="mean")
    # (runs begin elsewhere: fp32 rounding, and at times another bf16)
    close(h[:, tail], alone.double(), 2 * HALF["bf16"])
    close(hT, aT.double(), 2.0 ** -24, 2 * TOL32 * alone.double().abs().amax((0, 1)))
    got = ops.gated_scan_backward(x, gate, h, dh=dh, mix="mean")
    for part_of in (slice(0, part), tail):
        a = [v[:, part_of].clone() for v in (x, gate, h, dh)]
        want = ops.gated_scan_backward(a[0], a[1], a[2], dh=a[3], mix="mean")
        size = 4 * HALF["bf16"] * a[2].double().abs().amax((0, 1))
        close(got["x"][:, part_of], want["x"].double(), 2 * HALF["bf16"])
        # (the states are recomputed from other rows of h)
        close(got["gate"][:, part_of], want["gate"].double(), 2 * HALF["bf16"], size * want["x"].double().abs().amax((0, 1)))
