"""Linear attention with a decay per head where one head's, one row's or one
operand's size would hide another's: each head against its own size, values
whose scaled forms leave fp32, scores that overflow where the mask hides them.

Tolerances, normwise over the part that is compared.  fp32: 2e-5, as for whole
tensors (sums of a few hundred products).  bf16: the score, the copy of the
state and the output each round by up to 2^-9 of their own terms, which sum to
the output with mixed signs: 3 * 2^-9 = 6e-3, and 1e-2 with the terms that sum
to a little more.  The fp32 states: 2e-5 in both.
"""
import itertools

import pytest
import torch

from preconditioned_delta_rule_phase1_gb300 import build as osdn_build
from preconditioned_delta_rule_phase1_gb300 import ops
from tests._util import rel_err
from tests.test_decay_attn_gpu import STATE_TOL, TOL, WIDTHS, autograd, backward, forward, inputs, recurrence

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    osdn_build.build()
    ops.lib()


def each_head(got, ref, tol, what, rows=(0,)):
    """Every head by itself, over all tokens and over those from each of `rows` on (the
    first tokens' share of S0 would set the scale of a head that forgets at once)."""
    for h, t in itertools.product(range(ref.shape[1]), rows):
        if ref.dim() == 4 and t < ref.shape[2]:
            assert rel_err(got[:, h, t:], ref[:, h, t:].cpu()) < tol, (what, h, t)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("K,V", WIDTHS)
def test_each_head_of_the_outputs(io, K, V):
    for T, s0 in itertools.product([1, 2, 33, 64, 129, 257, 385], [False, True]):
        x = inputs(2, 7, T, K, V, io, seed=3 * T + K, s0=s0)
        o, ST = forward(x)
        ro, rS = recurrence(x["q"], x["k"], x["v"], x["decay"], x["S0"])
        each_head(o, ro, TOL[io], ("o", T, s0), rows=(0, 2, 128))
        each_head(ST, rS, STATE_TOL, ("ST", T, s0))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,T,K,V", [(1, 7, 3001, 128, 128), (1, 7, 2050, 64, 128), (40, 7, 130, 64, 64),
                                       (3, 7, 1111, 128, 64)])
def test_each_head_of_cut_sequences(io, B, H, T, K, V):
    x = inputs(B, H, T, K, V, io, seed=T)
    o, ST = forward(x)
    ro, rS = recurrence(x["q"], x["k"], x["v"], x["decay"], x["S0"])
    each_head(o, ro, TOL[io], "o", rows=(0, 2, 128, T // 2))
    each_head(ST, rS, STATE_TOL, "ST")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("K,V", WIDTHS)
def test_each_head_of_the_gradients(io, K, V):
    for (B, T), s0 in itertools.product([(2, 33), (2, 129), (1, 1030), (20, 70)], [False, True]):
        x = inputs(B, 7, T, K, V, io, seed=T + V + 1, s0=s0)
        got, ref = backward(x), autograd(x)
        for n in ("q", "k", "v"):
            each_head(got[n], ref[n], TOL[io], (n, B, T, s0), rows=(0, 2))
            if T > 2:   # the last tokens' share of dS_T
                each_head(got[n][:, :, :-2], ref[n][:, :, :-2], TOL[io], (n, B, T, s0, "but the last"))
        if s0:
            each_head(got["S0"], ref["S0"], STATE_TOL, ("S0", B, T))


LARGE = {"v": 1e33, "k": 1e33, "q": 1e35, "S0": 1e35, "do": 1e33, "dST": 1e35, "one token": 1e33}


@pytest.mark.parametrize("what", sorted(LARGE))
@pytest.mark.parametrize("B,H,T", [(2, 4, 150), (1, 4, 700)])
def test_large_values_in_fp32(what, B, H, T):
    # the recurrence is finite, so no scaled form of it may leave fp32's range
    x = inputs(B, H, T, 64, 128, "f32", seed=T, decay=torch.tensor([0.07, 0.3, 0.9, 0.999]))
    if what == "one token":
        x["v"][:, :, T // 2] *= LARGE[what]
    else:
        x[what] *= LARGE[what]
    if what in ("do", "dST"):
        x["S0"] *= 0.0
    else:
        o, ST = forward(x)
        ro, rS = recurrence(x["q"], x["k"], x["v"], x["decay"], x["S0"])
        each_head(o, ro, TOL["f32"], "o", rows=(0, T // 2))
        each_head(ST, rS, STATE_TOL, "ST")
        x["dST"] *= 0.0
    got, ref = backward(x), autograd(x)
    for n in ("q", "k", "v"):
        each_head(got[n], ref[n], TOL["f32"], n)
    each_head(got["S0"], ref["S0"], STATE_TOL, "S0")


@pytest.mark.parametrize("T", [100, 300, 2100])
def test_scores_that_overflow_behind_the_mask(T):
    # early queries times late keys exceed fp32, but no token reads a later key
    at = 71
    x = inputs(1, 3, T, 128, 64, "bf16", seed=T, decay=torch.tensor([0.9, 0.99, 1.0]))
    x["q"][:, :, :at] *= 1e25
    x["k"][:, :, at:] *= 1e25
    o, ST = forward(x)
    ro, rS = recurrence(x["q"], x["k"], x["v"], x["decay"], x["S0"])
    got, ref = backward(x), autograd(x)
    for part in (slice(0, at), slice(at, T)):
        each_head(o[:, :, part], ro[:, :, part], TOL["bf16"], ("o", part))
        for n in ("q", "k", "v"):
            each_head(got[n][:, :, part], ref[n][:, :, part], TOL["bf16"], (n, part))
    each_head(ST, rS, STATE_TOL, "ST")
    each_head(got["S0"], ref["S0"], STATE_TOL, "S0")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_step_and_gradients_in_a_graph(io):
    x = inputs(1, 4, 700, 128, 128, io, seed=8, decay=torch.tensor([0.99, 0.999, 1.0, 0.9]))
    one = {n: x[n][:, :, 0].contiguous() for n in "qkv"}
    S, o = x["S0"].clone(), torch.empty_like(one["v"])
    ws = ops.Workspace()
    step = lambda: ops.decay_attn_step(one["q"], one["k"], one["v"], x["decay"], S, o=o, workspace=ws)  # noqa: E731
    step()
    backward(x, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
        g = backward(x, ws)
    for t in (one["v"], x["v"], x["S0"]):
        t.mul_(-1.0)
    S.copy_(x["S0"])
    graph.replay()
    torch.cuda.synchronize()
    S2 = x["S0"].clone()
    o2 = ops.decay_attn_step(one["q"], one["k"], one["v"], x["decay"], S2)
    want = backward(x)
    assert torch.equal(o, o2) and torch.equal(S, S2)
    assert all(torch.equal(g[n], want[n]) for n in want)
    assert ws.status() == 0
