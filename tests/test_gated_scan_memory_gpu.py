"""Memories longer than fp32 can say of a: the product of many gates near 1, and the
state that it carries, against closed forms and the token recurrence in 64 bits.

With a constant gate, a = sigmoid(gate) and b = 1 - a,
    h_t = a^t h_0 + w x (1 - a^t) / b,     dh_0 = a^T dhT.

Tolerance.  Let L = T b be how far a state decays (as a power of e).  b itself is
within 2 ulp of an exponential and of a quotient, and its argument g log2 e rounds by
2^-24 of itself: 4.2e-7 + 7.3e-8 g, 1.9e-6 at most here.  16 tokens' product adds 32
roundings of 2^-25 to 1 - A, 1e-6.  A run that decays by 1/128 or more has its A
rounded, 2^-25 128 = 3.8e-6 of the decay, and so have eight of them; one that decays
less keeps 1e-6.  Together 1.1e-5 L of the state.  The state itself is a sum in fp32 of
what runs of at least 64 tokens (8 of 8 warps) leave of it and add, T / 64 sums that with a constant input
may all round to the same side: 2^-24 T / 64.  Within a run of at most 16 tokens each is
rounded as any fp32 recurrence does: 16 roundings of 2^-23.
Where a itself was multiplied 2^16 times and more, each time rounded to a multiple of
2^-24, these came to 1e-3 and, from a gate of 16.7 on, to all of the decay.
"""
import pytest
import torch

from preconditioned_delta_rule_phase1_gb300 import build as osdn_build
from preconditioned_delta_rule_phase1_gb300 import ops

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
GATES = [7.0, 8.0, 9.0, 9.5, 10.0, 11.0, 12.0, 13.0, 14.0, 15.0, 16.0, 17.0, 18.0, 20.0]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    osdn_build.build()
    ops.lib()


def tolerance(T, b):
    return 1.1e-5 * T * b + T / 64 * 2.0 ** -24 + 16 * 2.0 ** -23


def closed(T, mix):
    """log a, b, w of the gates (exact in bf16), and a^t [T+1,C]."""
    g = torch.tensor(GATES, dtype=torch.float64, device="cuda")
    b = torch.sigmoid(-g)
    w = {"sum": torch.ones_like(b), "mean": b, "unit": (b * (2 - b)).sqrt()}[mix]
    t = torch.arange(T + 1, dtype=torch.float64, device="cuda")[:, None]
    return b, w, t * torch.log1p(-b)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1000, 65536, 262147])
def test_a_state_decays_by_the_product_of_its_gates(io, T):
    b, _, log = closed(T, "sum")
    C = len(GATES)
    x = torch.zeros(1, T, C, dtype=DT[io], device="cuda")
    gate = torch.tensor(GATES, device="cuda").to(DT[io]).expand(1, T, C).contiguous()
    one = torch.ones(1, C, device="cuda")
    want = log.exp()
    tol, small = tolerance(T, b), 2.0 ** -100   # (a state that has decayed so far may be anything as small)
    off = lambda got, ref, tol: float(((got.double() - ref).abs() / (tol * ref + small)).max())  # noqa: E731
    h, hT = ops.gated_scan(x, gate, one, mix="sum")
    assert off(hT[0], want[-1], tol) < 1
    assert off(h[0], want[1:], tol + HALF[io]) < 1
    g = ops.gated_scan_backward(x, gate, h, one, dh=x, dhT=one, mix="sum")
    assert off(g["h0"][0], want[-1], tol) < 1
    # dx_t = R_t = a^(T - t)
    assert off(g["x"][0].flip(0), want[:-1], tol + HALF[io]) < 1


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("mix", ["sum", "mean", "unit"])
@pytest.mark.parametrize("T", [65536, 1 << 20])
def test_a_constant_input_fills_the_memory(io, mix, T):
    b, w, log = closed(T, mix)
    C = len(GATES)
    x = torch.ones(1, T, C, dtype=DT[io], device="cuda")
    gate = torch.tensor(GATES, device="cuda").to(DT[io]).expand(1, T, C).contiguous()
    h, hT = ops.gated_scan(x, gate, mix=mix)
    want = w * -torch.expm1(log[1:]) / b
    tol = tolerance(T, b) + 4e-6   # (w is off by as much as b, and each run's own sum by 16 roundings)
    off = (hT[0].double() / want[-1] - 1).abs() / tol
    assert bool((off < 1).all()), off.tolist()
    assert bool(((h[0].double() / want - 1).abs() < tol + HALF[io]).all())


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("mix", ["sum", "mean", "unit"])
def test_nearly_open_gates_over_60000_tokens(io, mix):
    """Gates from 14 to 20 and inputs that differ from token to token; the single-token call goes on from
    where the prompt stops."""
    T, C = 60000, 65
    g = torch.Generator().manual_seed(3)
    x = (1 + torch.randn(1, T, C, generator=g)).to(DT[io]).cuda()
    gate = (14 + 6 * torch.rand(C, generator=g) + 0.1 * torch.randn(1, T, C, generator=g)).to(DT[io]).cuda()
    h0 = (100 * torch.randn(1, C, generator=g)).cuda()
    gd = gate[0].double()
    a, b = torch.sigmoid(gd), torch.sigmoid(-gd)
    w = {"sum": torch.ones_like(b), "mean": b, "unit": (b * (1 + a)).sqrt()}[mix]
    wx, s = w * x[0].double(), h0[0].double()
    most = s.abs()
    for t in range(T):
        s = torch.addcmul(wx[t], a[t], s)
        most = torch.maximum(most, s.abs())
    _, hT = ops.gated_scan(x, gate, h0, mix=mix)
    tol = (tolerance(T, b.amax(0)) + 4e-6) * most
    off = (hT[0].double() - s).abs() / tol
    assert bool((off < 1).all()), float(off.max())
    cut = T - 2
    _, state = ops.gated_scan(x[:, :cut].contiguous(), gate[:, :cut].contiguous(), h0, mix=mix)
    for t in range(cut, T):
        y = ops.gated_scan_step(x[:, t].clone(), gate[:, t].clone(), state, mix=mix)
    off = (state[0].double() - s).abs() / tol
    assert bool((off < 1).all()), float(off.max())
    assert torch.equal(y, state.to(DT[io]))
