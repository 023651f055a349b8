"""Group norm with an activation (osdn_group_norm and its gradients) against
the formula in 64 bits.

Tolerances, normwise: fp32 arithmetic on at most 512 values a group and on
fp32 sums over the tokens, 2e-5; bf16 outputs round once, 2^-9 of their own
size, 4e-3 of the largest.
"""
import itertools

import pytest
import torch

from preconditioned_delta_rule_phase1_gb300 import build as osdn_build
from preconditioned_delta_rule_phase1_gb300 import ops
from tests._util import rel_err

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
TOL = {"f32": 2e-5, "bf16": 4e-3}
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    osdn_build.build()
    ops.lib()


def act64(u, act):
    return {"none": u, "silu": u / (1 + torch.exp(-u)), "sigmoid": 1 / (1 + torch.exp(-u))}[act]


def formula(x, weight, bias, gate, groups, act, first):
    """y in 64 bits; x [B,G,T,D] (first) or [B,T,C]."""
    x = x.transpose(1, 2) if first else x.reshape(*x.shape[:2], groups, -1)
    m = x.mean(-1, keepdim=True)
    z = ((x - m) / ((x - m).square().mean(-1, keepdim=True) + EPS).sqrt()).flatten(2)
    z = z if weight is None else z * weight
    z = z if bias is None else z + bias
    return act64(z, act) if gate is None else z * act64(gate, act)


def inputs(B, G, T, D, io, first, affine, gated, seed, mean=0.3):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = n(*((B, G, T, D) if first else (B, T, G * D))) + mean
    return {"x": x.to(DT[io]).cuda(), "weight": (1 + 0.2 * n(G * D)).cuda() if affine else None,
            "bias": (0.2 * n(G * D)).cuda() if affine else None,
            "gate": n(B, T, G * D).to(DT[io]).cuda() if gated else None,
            "dy": n(B, T, G * D).to(DT[io]).cuda()}


SHAPES = [(1, 1, 1, 8), (2, 3, 5, 16), (1, 2, 33, 24), (3, 5, 17, 64), (2, 16, 70, 128), (1, 3, 9, 200),
          (2, 2, 31, 256), (1, 2, 13, 264), (1, 1, 300, 512), (257, 1, 1, 40)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("act", ["none", "silu", "sigmoid"])
def test_matches_the_formula(io, first, act):
    ws = ops.Workspace()
    for (B, G, T, D), affine, gated in itertools.product(SHAPES, [True, False], [True, False]):
        t = inputs(B, G, T, D, io, first, affine, gated, seed=D + T)
        kw = dict(weight=t["weight"], bias=t["bias"], gate=t["gate"], groups=G, act=act, eps=EPS)
        wide = {n: None if v is None else v.double().requires_grad_(n != "dy") for n, v in t.items()}
        ref = formula(wide["x"], wide["weight"], wide["bias"], wide["gate"], G, act, first)
        y = ops.group_norm(t["x"], **kw)
        assert rel_err(y, ref.detach().cpu()) < TOL[io], (B, G, T, D, affine, gated)
        names = [n for n in ("x", "weight", "bias", "gate") if t[n] is not None]
        want = dict(zip(names, torch.autograd.grad(ref, [wide[n] for n in names], wide["dy"])))
        got = ops.group_norm_backward(t["x"], t["dy"], workspace=ws, **kw)
        assert sorted(got) == sorted(names)
        for n in names:
            tol = 2e-5 if n in ("weight", "bias") else TOL[io]
            # where the group has few channels dx is a small rest of large terms
            # (dx = 0 for one channel's worth of freedom): against the terms' size
            size = max(1.0, float((wide["dy"].abs().max()) / want[n].abs().max())) if n == "x" else 1.0
            assert rel_err(got[n], want[n].cpu()) < tol * size, (n, B, G, T, D, affine, gated)


def test_gradients_match_differences():
    t = inputs(2, 3, 7, 64, "f32", True, True, True, seed=3)
    kw = dict(groups=3, act="silu", eps=EPS)
    args = {n: t[n] for n in ("x", "weight", "bias", "gate")}
    got = ops.group_norm_backward(t["x"], t["dy"], t["weight"], t["bias"], t["gate"], **kw)
    g = torch.Generator(device="cuda").manual_seed(1)
    h = 2.0 ** -7
    for n in args:
        u = torch.randn(args[n].shape, generator=g, device="cuda")
        f = [float((ops.group_norm(**{**args, n: args[n] + s * u}, **kw).double() * t["dy"].double()).sum())
             for s in (h, -h)]
        want, have = (f[0] - f[1]) / (2 * h), float((got[n].double() * u.double()).sum())
        # central differences: h^2 of the third derivative (order one a term) over sqrt(n) terms
        scale = float((got[n].double() * u.double()).square().sum().sqrt())
        assert abs(want - have) < 2e-2 * scale, (n, want, have)


def test_constant_groups_and_large_means():
    x = torch.full((2, 3, 4, 64), 7.0, device="cuda")
    bias = torch.randn(192, device="cuda")
    y = ops.group_norm(x, None, bias, act="none")
    assert torch.equal(y, bias.expand(2, 4, 192))   # no spread: x^ = 0
    # a mean a thousand times the spread: fp32 holds 7 digits, 4 are left of the spread's
    x = (1000.0 + torch.randn(2, 3, 4, 64, generator=torch.Generator().manual_seed(1))).cuda()
    ref = formula(x.double(), None, None, None, 3, "none", True)
    assert rel_err(ops.group_norm(x), ref.cpu()) < 2e-5


def test_extreme_gates():
    x = torch.randn(1, 2, 3, 8, device="cuda")
    z = ops.group_norm(x)
    gate = torch.tensor([-200.0, 200.0, -88.0, 0.0], device="cuda").repeat(12).reshape(1, 3, 16).contiguous()
    want = z.double() * act64(gate.double().clamp(-100, 300), "silu")
    got = ops.group_norm(x, gate=gate, act="silu")
    assert torch.isfinite(got).all() and rel_err(got, want.cpu()) < 2e-5


def test_empty_and_repeatable():
    w = torch.ones(32, device="cuda")
    x = torch.empty(2, 0, 32, device="cuda")
    assert ops.group_norm(x, w, w, groups=2).shape == (2, 0, 32)
    g = ops.group_norm_backward(x, torch.empty(2, 0, 32, device="cuda"), w, w, groups=2)
    assert not g["weight"].any() and not g["bias"].any()
    t = inputs(3, 4, 999, 128, "bf16", True, True, True, seed=6)
    run = lambda: ops.group_norm_backward(t["x"], t["dy"], t["weight"], t["bias"], t["gate"], act="silu")  # noqa: E731
    a, b = run(), run()
    assert all(torch.equal(a[n], b[n]) for n in a)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        c = run()
    side.synchronize()
    assert all(torch.equal(a[n], c[n]) for n in a)
