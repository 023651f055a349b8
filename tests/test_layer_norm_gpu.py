"""Layer norm with the residual stream's addition (osdn_layer_norm and its
gradients) against the formula in 64 bits.

Tolerances: an I/O rounding is off by at most half a step of the value (bf16
2^-8, fp32 2^-24); fp32 statistics over up to 16384 values, summed in lanes of at
most some dozens and then pairwise, are within 2e-6 relative, and so are the
normed values: 1e-5 of the row's largest covers the few products behind them.
The gradients' mean terms cancel against u: 1e-5 of the row's largest |u| over
the standard deviation.  dweight and dbias add up rows: 1e-5 of the sum of the
terms' sizes, each with its row's largest normed value.
"""
import pytest
import torch

from preconditioned_delta_rule_phase1_gb300 import build as osdn_build
from preconditioned_delta_rule_phase1_gb300 import ops

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    osdn_build.build()
    ops.lib()


def inputs(shape, io, seed, mean=0.3):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    C = shape[-1]
    return {"x": (n(*shape) + mean).to(DT[io]).cuda(), "residual": n(*shape).to(DT[io]).cuda(),
            "weight": (1 + 0.2 * n(C)).cuda(), "bias": (0.2 * n(C)).cuda(), "dy": n(*shape).to(DT[io]).cuda(),
            "ds": n(*shape).to(DT[io]).cuda()}


def normed64(s):
    m = s.mean(-1, keepdim=True)
    r = 1 / ((s - m).square().mean(-1, keepdim=True) + EPS).sqrt()
    return (s - m) * r, r


def row(v):
    return v.abs().amax(-1, keepdim=True)


def within(got, ref, bound, what=""):
    assert got.shape == ref.shape, what
    off = (got.double() - ref).abs() - bound
    assert not ref.numel() or bool((off <= 0).all()), (what, float(off.max()))


def check(t, io, affine, residual, what="", ws=None):
    d = {k: v.double() for k, v in t.items()}
    w, b = (t["weight"], t["bias"]) if affine else (None, None)
    w64, b64 = (d["weight"], d["bias"]) if affine else (torch.ones_like(d["weight"]), torch.zeros_like(d["bias"]))
    s = d["x"] + d["residual"] if residual else d["x"]
    xh, r = normed64(s)
    y64 = xh * w64 + b64
    if residual:
        y, stream = ops.layer_norm(t["x"], w, b, residual=t["residual"], eps=EPS)
        within(stream, s, HALF[io] * s.abs() + 2.0 ** -23 * s.abs(), ("s", what))
    else:
        y = ops.layer_norm(t["x"], w, b, eps=EPS)
        stream = t["x"]
    # fp32 rounding of s (with a residual) is relative to s, and the norm divides by the spread
    tol = 1e-5 * (row(xh) * w64.abs() + b64.abs()) + 2.0 ** -23 * row(s) * r * w64.abs()
    within(y, y64, HALF[io] * y64.abs() + tol, ("y", what))
    # gradients at what was normed, as it was stored
    xh, r = normed64(stream.double())
    u = d["dy"] * w64
    dx = r * (u - u.mean(-1, keepdim=True) - xh * (u * xh).mean(-1, keepdim=True))
    tol = 1e-5 * r * row(u) * (1 + row(xh))
    if residual:
        dx = dx + d["ds"]
    g = ops.layer_norm_backward(stream, t["dy"], w, b, ds=t["ds"] if residual else None, eps=EPS, workspace=ws)
    assert sorted(g) == (["bias", "weight", "x"] if affine else ["x"])
    within(g["x"], dx, HALF[io] * dx.abs() + tol, ("dx", what))
    if affine:
        rows = lambda v: v.reshape(-1, v.shape[-1]).sum(0)  # noqa: E731
        dy = d["dy"]
        within(g["weight"], rows(dy * xh), 1e-5 * rows(dy.abs() * row(xh)), ("dweight", what))
        within(g["bias"], rows(dy), 1e-5 * rows(dy.abs()), ("dbias", what))


WIDTHS = [2, 3, 7, 8, 31, 32, 33, 64, 100, 127, 128, 129, 255, 256, 264, 500, 512, 513, 690, 1000, 1023, 1024, 1025,
          1030, 2047, 2048, 2049, 2056, 4095, 4096, 4100, 5000, 8191, 8192, 8200, 12000, 16383, 16384]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("residual", [False, True])
def test_widths(io, residual):
    ws = ops.Workspace()
    for i, C in enumerate(WIDTHS):
        for rows in ((1, 5, 37)[i % 3], 3):
            check(inputs((rows, C), io, seed=C), io, affine=i % 4 != 1, residual=residual, what=(rows, C), ws=ws)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,C", [(1, 2048), (151, 2048), (153, 64), (609, 1030), (1217, 129), (2500, 256),
                                    (5000, 2048), (300, 8192), (70001, 8), (3, 16384)])
def test_rows(io, rows, C):
    check(inputs((rows, C), io, seed=rows), io, True, True, (rows, C))
    check(inputs((rows, C), io, seed=rows + 1), io, True, False, (rows, C))


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_dimensions(io):
    for shape in ((40,), (2, 3, 40), (2, 1, 3, 5, 24)):
        check(inputs(shape, io, seed=1), io, True, True, shape)
    one = inputs((9, 1), io, seed=1)   # a single channel: x^ = 0
    y = ops.layer_norm(one["x"], one["weight"], one["bias"])
    assert torch.equal(y, one["bias"].to(DT[io]).expand_as(y))
    g = ops.layer_norm_backward(one["x"], one["dy"], one["weight"], one["bias"])
    # u - mean(u) = 0 but for two roundings of u, times 1 / sqrt(eps)
    within(g["x"], torch.zeros_like(one["x"]).double(),
           2.0 ** -23 * EPS ** -0.5 * (one["dy"].double() * one["weight"].double()).abs())
    assert not g["weight"].any()


@pytest.mark.parametrize("C", [64, 1000, 2048, 5000, 16384])
def test_constant_rows_and_large_means(C):
    x = torch.full((7, C), 7.0, device="cuda")
    bias = torch.randn(C, device="cuda")
    assert torch.equal(ops.layer_norm(x, None, bias), bias.expand(7, C))   # no spread: x^ = 0
    # a mean a thousand times the spread
    x = (1000.0 + torch.randn(7, C, generator=torch.Generator().manual_seed(1))).cuda()
    xh, _ = normed64(x.double())
    within(ops.layer_norm(x), xh, 1e-5 * row(xh))
    dy = torch.randn(7, C, device="cuda")
    u, (xh, r) = dy.double(), normed64(x.double())
    dx = r * (u - u.mean(-1, keepdim=True) - xh * (u * xh).mean(-1, keepdim=True))
    within(ops.layer_norm_backward(x, dy)["x"], dx, 1e-5 * row(u) * (1 + row(xh)) * r)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("C", [40, 513, 1000, 2048, 5000, 16384])
def test_a_first_value_far_from_the_others(io, C):
    """Sums are taken of differences to the row's first value: here it is no guide to the others."""
    t = inputs((9, C), io, seed=C)
    for r, far in enumerate((0.0, 3.0, 8.0, -20.0, 100.0, -3000.0, 1e6, 0.0, -40.0)):
        t["x"][r, 0] += far
        t["residual"][r, 0] = 0
    check(t, io, True, False, C)
    check(t, io, True, True, C)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_a_bad_row_stays_alone(io):
    t = inputs((9, 300), io, seed=2)
    want = ops.layer_norm(t["x"], t["weight"], t["bias"])
    gx = ops.layer_norm_backward(t["x"], t["dy"], t["weight"])["x"]
    t["x"][4, 17] = float("inf")
    t["x"][6, 0] = float("nan")
    got = ops.layer_norm(t["x"], t["weight"], t["bias"])
    gg = ops.layer_norm_backward(t["x"], t["dy"], t["weight"])["x"]
    keep = [0, 1, 2, 3, 5, 7, 8]
    assert torch.equal(got[keep], want[keep]) and torch.equal(gg[keep], gx[keep])
    assert got[6].isnan().all() and got[4].isnan().any() and gg[6].isnan().all()


@pytest.mark.parametrize("C", [40, 1030])
def test_gradients_match_differences(C):
    t = inputs((6, C), "f32", seed=3)
    s = t["x"] + t["residual"]
    got = ops.layer_norm_backward(s, t["dy"], t["weight"], t["bias"], ds=t["ds"])
    args = {n: t[n] for n in ("x", "weight", "bias", "residual")}
    g = torch.Generator(device="cuda").manual_seed(1)
    step = 2.0 ** -7

    def loss(**kw):
        y, s = ops.layer_norm(**{**args, **kw}, eps=EPS)
        return float((y.double() * t["dy"].double()).sum() + (s.double() * t["ds"].double()).sum())
    for n in args:
        u = torch.randn(args[n].shape, generator=g, device="cuda")
        want = (loss(**{n: args[n] + step * u}) - loss(**{n: args[n] - step * u})) / (2 * step)
        terms = got["x" if n == "residual" else n].double() * u.double()
        # central differences: step^2 of the third derivative (order one a term)
        assert abs(want - float(terms.sum())) < 1e-2 * float(terms.square().sum().sqrt()), n


def test_optional_arguments_and_empty():
    t = inputs((48, 130), "bf16", seed=5)
    both = ops.layer_norm_backward(t["x"], t["dy"], t["weight"], t["bias"])
    only = ops.layer_norm_backward(t["x"], t["dy"], None, t["bias"])
    assert sorted(only) == ["bias", "x"] and torch.equal(only["bias"], both["bias"])
    only = ops.layer_norm_backward(t["x"], t["dy"], t["weight"])
    assert sorted(only) == ["weight", "x"] and torch.equal(only["weight"], both["weight"])
    assert torch.equal(only["x"], both["x"])
    y = torch.full((3, 48, 130), 7.0, dtype=torch.bfloat16, device="cuda")
    s = y.clone()
    ops.layer_norm(t["x"], t["weight"], residual=t["residual"], y=y[1], s=s[1])
    assert bool((y[::2] == 7).all()) and bool((s[::2] == 7).all())
    e = torch.empty(0, 32, device="cuda")
    w = torch.ones(32, device="cuda")
    assert ops.layer_norm(e, w, w).shape == (0, 32)
    g = ops.layer_norm_backward(e, e, w, w)
    assert not g["weight"].any() and not g["bias"].any() and g["x"].shape == (0, 32)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,C", [(3, 2048), (2000, 1030), (900, 4096)])
def test_repeatable_elsewhere_and_in_a_graph(io, rows, C):
    t = inputs((rows, C), io, seed=6)
    ws = ops.Workspace()

    def run(stream=None, ws=ws):
        y, s = ops.layer_norm(t["x"], t["weight"], t["bias"], residual=t["residual"], stream=stream)
        g = ops.layer_norm_backward(s, t["dy"], t["weight"], t["bias"], ds=t["ds"], workspace=ws, stream=stream)
        return [y, s, g["x"], g["weight"], g["bias"]]
    want = run()
    ws.buf[256:] = 0x5a   # whatever an earlier call has left
    assert all(torch.equal(a, b) for a, b in zip(run(), want))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = run(side, ops.Workspace(stream=side))
    here = run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(torch.equal(a, b) for a, b in zip(here, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    t["x"].mul_(-2.0)
    t["dy"].add_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, run()))


def test_offsets_past_32_bits():
    """More than 2^31 elements a tensor: the last rows are what they are alone."""
    rows, C, part = 1100003, 1990, 300
    assert rows * C > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(1)
    x, r, dy = (torch.empty(rows, C, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(3))
    w = torch.randn(C, generator=g, device="cuda")
    y, s = ops.layer_norm(x, w, residual=r)
    dx = ops.layer_norm_backward(s, dy, w, ds=r)["x"]
    tail = slice(rows - part, rows)
    a = [v[tail].clone() for v in (x, r, s, dy)]
    want, sw = ops.layer_norm(a[0], w, residual=a[1])
    assert torch.equal(s[tail], sw)
    # (rows are cut otherwise where they are few: fp32 rounding, and at times another bf16)
    within(y[tail], want.double(), 2 * HALF["bf16"] * want.double().abs() + 1e-5 * row(want.double()))
    want = ops.layer_norm_backward(a[2], a[3], w, ds=a[1])["x"]
    within(dx[tail], want.double(), 2 * HALF["bf16"] * want.double().abs() + 1e-5 * row(want.double()))
