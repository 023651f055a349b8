"""Cases of the gated recurrent layer: its recurrence with a gate for every token and
channel (whole prompts, single tokens, gradients), and the layer norm in front of it,
with the residual stream's addition (forward, gradients).

Recurrence, per sequence and channel, from h_0, with a_t = sigmoid(gate_t):
    h_t = a_t h_{t-1} + w(a_t) x_t
    w(a) = 1 (mix "sum"), 1 - a ("mean") or sqrt(1 - a^2) ("unit")
Layer norm, per token over its C channels:
    s = x + residual (or x),    y = weight (s - mean) / sqrt(var + eps) + bias

``own`` false: the plain forms below, elementary torch operations in fp32.
``own`` true: the library's calls.
"""
import math

import torch

own = False

BLOCK = 256          # tokens a block of the plain recurrence
EPS = 1e-5
DOCUMENT = 3001      # mean length of the documents packed into one sequence
DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


# ----------------------------------------------------------------------- cases
def listed():
    return [
        # a user's next turn in fp32, read on from a state: a parity run, few and odd channels
        {"name": "scan_turn_f32", "op": "scan", "io": "f32", "B": 2, "T": 777, "C": 501, "mix": "sum",
         "h0": True, "docs": False},
        # the 340M-class layer over a batch of prompts
        {"name": "scan_batch", "op": "scan", "io": "bf16", "B": 8, "T": 2048, "C": 1024, "mix": "unit",
         "h0": False, "docs": False},
        # the 1.3B-class layer over one long sequence of packed documents, read on from a state
        {"name": "scan_long", "op": "scan", "io": "bf16", "B": 1, "T": 65536, "C": 2048, "mix": "mean",
         "h0": True, "docs": True},
        # one user's next token: latency
        {"name": "step_one", "op": "step", "io": "bf16", "B": 1, "C": 2048, "mix": "mean"},
        # a full serving batch's next token
        {"name": "step_batch", "op": "step", "io": "bf16", "B": 256, "C": 2048, "mix": "unit"},
        # truncated back-propagation over an odd piece, with both states' gradients
        {"name": "scan_train_odd", "op": "scan_train", "io": "bf16", "B": 3, "T": 1037, "C": 690,
         "mix": "unit", "h0": True, "docs": False},
        # the 1.3B-class layer's training step over packed documents
        {"name": "scan_train_long", "op": "scan_train", "io": "bf16", "B": 2, "T": 8192, "C": 2048,
         "mix": "mean", "h0": False, "docs": True},
        # the norm in front of step_batch
        {"name": "norm_token", "op": "norm", "io": "bf16", "B": 256, "T": 1, "C": 2048, "residual": True},
        # a parity run in fp32 at an odd width
        {"name": "norm_odd_f32", "op": "norm", "io": "f32", "B": 2, "T": 777, "C": 1003, "residual": False},
        # the norm in front of the 1.3B-class layer
        {"name": "norm_prompt", "op": "norm", "io": "bf16", "B": 2, "T": 8192, "C": 2048, "residual": True},
        # its gradients at an odd length and width, no residual stream
        {"name": "norm_train_odd", "op": "norm_train", "io": "bf16", "B": 3, "T": 2731, "C": 1030,
         "residual": False},
        # the 1.3B-class layer's training step, the residual stream's gradient added on the way
        {"name": "norm_train_long", "op": "norm_train", "io": "bf16", "B": 2, "T": 8192, "C": 2048,
         "residual": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan", "scan", "step", "scan_train", "scan_train", "norm", "norm_train"])
    io = rng.choice(["bf16", "bf16", "bf16", "f32"])
    mix = rng.choice(["sum", "mean", "unit"])
    if op == "step":
        return {"op": op, "io": io, "B": _log(rng, 1, 256), "C": _log(rng, 32, 1024 if io == "f32" else 2048),
                "mix": mix}
    # elements bounded by the largest listed case of the op (half of it in fp32)
    most = (1 << (27 if op == "scan" else 25)) >> (1 if io == "f32" else 0)
    if op in ("scan", "scan_train"):
        C = _log(rng, 32, 4096)
        T = _log(rng, 1, min(65536 if op == "scan" else 16384, most // C))
        B = _log(rng, 1, max(1, min(8, most // (C * T))))
        return {"op": op, "io": io, "B": B, "T": T, "C": C, "mix": mix, "h0": rng.random() < 0.5,
                "docs": rng.random() < 0.5}
    C = _log(rng, 32, 16384)
    T = _log(rng, 1, min(8192, most // C))
    B = _log(rng, 1, max(1, min(256, most // (C * T))))
    return {"op": op, "io": io, "B": B, "T": T, "C": C, "residual": rng.random() < 0.5}


# ---------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    op, B, C, dt = case["op"], case["B"], case["C"], DTYPE[case["io"]]
    s = {"case": case}
    if op in ("norm", "norm_train"):
        T = case["T"]
        # a stream whose channels differ in mean and size, as trained ones do
        size, mean = torch.exp(0.5 * normal(C)), 0.3 * normal(C)
        s["x"] = (normal(B, T, C) * size + mean).to(dt)
        s["weight"], s["bias"] = 1.0 + 0.1 * normal(C), 0.1 * normal(C)
        if op == "norm":
            s["residual"] = normal(B, T, C).to(dt) if case["residual"] else None
        else:
            s["dy"] = normal(B, T, C).to(dt)
            s["ds"] = normal(B, T, C).to(dt) if case["residual"] else None
        return s
    shape = (B, C) if op == "step" else (B, case["T"], C)
    s["x"] = normal(*shape).to(dt)
    # memories from about 3 tokens to about 1000, one a channel, moved by the token
    gate = 1.0 + 6.0 * torch.rand(C, generator=g, device="cuda") + normal(*shape)
    if case.get("docs"):   # a document's first token forgets the state: sigmoid(-inf) = 0
        first = torch.rand(B, case["T"], generator=g, device="cuda") < 1.0 / DOCUMENT
        gate = torch.where(first[..., None], -math.inf, gate)
    s["gate"] = gate.to(dt)
    if op == "step":
        s["h"] = normal(B, C)
        return s
    s["h0"] = normal(B, C) if case["h0"] else None
    if op == "scan_train":
        s["h"] = _scan(s)["h"]   # what the forward pass has left
        s["dh"] = normal(*shape).to(dt)
        s["dhT"] = normal(B, C) if case["h0"] else None
    return s


# ----------------------------------------------------------------- plain forms
def _weights(s):
    """a and w(a) in fp32; 1 - a as sigmoid(-gate), which keeps its digits near a = 1."""
    gate, mix = s["gate"].float(), s["case"]["mix"]
    a, b = torch.sigmoid(gate), torch.sigmoid(-gate)
    return a, torch.ones_like(a) if mix == "sum" else b if mix == "mean" else (b * (1.0 + a)).sqrt()


def _recur(a, b, h):
    """h_t = a_t h_{t-1} + b_t over dimension 1: every block from zero, all blocks at once,
    then the states between blocks, then their parts."""
    B, T, C = a.shape
    n = -(-T // BLOCK)
    L = -(-T // n)
    if n * L != T:
        a = torch.cat([a, a.new_ones(B, n * L - T, C)], 1)
        b = torch.cat([b, b.new_zeros(B, n * L - T, C)], 1)
    a, b = (x.reshape(B, n, L, C) for x in (a, b))
    out, power = torch.empty_like(a), torch.empty_like(a)
    x, p = torch.zeros_like(a[:, :, 0]), torch.ones_like(a[:, :, 0])
    for i in range(L):
        x = a[:, :, i] * x + b[:, :, i]
        p = p * a[:, :, i]
        out[:, :, i] = x
        power[:, :, i] = p
    start = []
    for j in range(n):
        start.append(h)
        h = power[:, j, -1] * h + out[:, j, -1]
    out += power * torch.stack(start, 1)[:, :, None]
    return out.reshape(B, n * L, C)[:, :T], h


def _start(s):
    return torch.zeros_like(s["x"][:, 0], dtype=torch.float32) if s["h0"] is None else s["h0"]


def _scan(s):
    a, w = _weights(s)
    h, hT = _recur(a, w * s["x"].float(), _start(s))
    return {"h": h.to(s["x"].dtype), "hT": hT}


def _scan_train(s):
    a, w = _weights(s)
    x, dh, mix, dt = s["x"].float(), s["dh"].float(), s["case"]["mix"], s["x"].dtype
    h, _ = _recur(a, w * x, _start(s))
    before = torch.cat([_start(s)[:, None], h[:, :-1]], 1)
    if s["dhT"] is not None:
        dh = dh.clone()
        dh[:, -1] += s["dhT"]
    # R_t = dh_t + a_{t+1} R_{t+1}: the same recurrence from the end
    later = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    R, _ = _recur(later.flip(1), dh.flip(1), torch.zeros_like(a[:, 0]))
    R = R.flip(1)
    b = torch.sigmoid(-s["gate"].float())
    da = a * b * before
    if mix == "mean":
        da = a * b * (before - x)
    if mix == "unit":   # w' = -a / w, and a (1 - a) a / w = a^2 sqrt((1 - a) / (1 + a))
        da = da - a * a * (b / (1.0 + a)).sqrt() * x
    out = {"x": (w * R).to(dt), "gate": (R * da).to(dt)}
    if s["h0"] is not None:
        out["h0"] = a[:, 0] * R[:, 0]
    return out


def _step(s):
    a, w = _weights(s)
    h = s["h"].mul_(a).add_(w * s["x"].float())
    return {"y": h.to(s["x"].dtype), "h": s["h"]}


def _normed(s):
    m = s.mean(-1, keepdim=True)
    r = ((s - m).square().mean(-1, keepdim=True) + EPS).rsqrt()
    return (s - m) * r, r


def _norm(s):
    x = s["x"].float()
    if s["residual"] is not None:
        x = x + s["residual"].float()
    y = (_normed(x)[0] * s["weight"] + s["bias"]).to(s["x"].dtype)
    return {"y": y} if s["residual"] is None else {"y": y, "s": x.to(s["x"].dtype)}


def _norm_train(s):
    xh, r = _normed(s["x"].float())
    dy = s["dy"].float()
    t = dy * s["weight"]
    dx = r * (t - t.mean(-1, keepdim=True) - xh * (t * xh).mean(-1, keepdim=True))
    if s["ds"] is not None:
        dx = dx + s["ds"].float()
    return {"x": dx.to(s["x"].dtype), "weight": (dy * xh).sum((0, 1)), "bias": dy.sum((0, 1))}


PLAIN = {"scan": _scan, "scan_train": _scan_train, "step": _step, "norm": _norm, "norm_train": _norm_train}


# ----------------------------------------------------------------------- a pass
def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return PLAIN[op](s)
    from preconditioned_delta_rule_phase1_gb300 import ops

    ws = s.get("ws")
    if ws is None:  # the workspace that a program keeps for its calls
        ws = s["ws"] = ops.Workspace()
    if op == "scan":
        h, hT = ops.gated_scan(s["x"], s["gate"], s["h0"], mix=case["mix"], workspace=ws)
        return {"h": h, "hT": hT}
    if op == "scan_train":
        # (in fp32 the plain recurrence may leave h as a slice; the call reads it densely)
        return ops.gated_scan_backward(s["x"], s["gate"], s["h"].contiguous(), s["h0"], dh=s["dh"],
                                       dhT=s["dhT"], mix=case["mix"], workspace=ws)
    if op == "step":
        return {"y": ops.gated_scan_step(s["x"], s["gate"], s["h"], mix=case["mix"]), "h": s["h"]}
    if op == "norm":
        if s["residual"] is None:
            return {"y": ops.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS)}
        y, stream = ops.layer_norm(s["x"], s["weight"], s["bias"], residual=s["residual"], eps=EPS)
        return {"y": y, "s": stream}
    return ops.layer_norm_backward(s["x"], s["dy"], s["weight"], s["bias"], ds=s["ds"], eps=EPS, workspace=ws)


# ------------------------------------------------------------------------- work
def work(case):
    op, B, C = case["op"], case["B"], case["C"]
    e = 4 if case["io"] == "f32" else 2
    n = B * case.get("T", 1) * C
    if op == "step":    # x, gate, y and the state both ways; an exponential counts as one
        return {"bytes": n * (3 * e + 8), "flops": 8 * n}
    if op == "scan":    # x, gate, h
        return {"bytes": 3 * n * e + 4 * B * C * (2 if case["h0"] else 1), "flops": 8 * n}
    if op == "scan_train":   # x, gate, dh, dx, dgate: the states can be had from x and gate
        return {"bytes": 5 * n * e + (12 * B * C if case["h0"] else 0), "flops": 18 * n}
    if op == "norm":
        return {"bytes": (4 if case["residual"] else 2) * n * e + 8 * C, "flops": 8 * n}
    return {"bytes": (4 if case["residual"] else 3) * n * e + 12 * C, "flops": 16 * n}


# ------------------------------------------------------------------------ 64 bits
def _mix64(gate, mix):
    """a, w(a) and d w / d gate."""
    a, forget = 1.0 / (1.0 + torch.exp(-gate)), 1.0 / (1.0 + torch.exp(gate))
    if mix == "sum":
        return a, torch.ones_like(a), torch.zeros_like(a)
    if mix == "mean":
        return a, forget, -a * forget
    return a, torch.sqrt(forget * (1.0 + a)), -a.square() * torch.sqrt(forget / (1.0 + a))


def _tokens64(a, b, h):
    """The recurrence token by token; [T,B,C] in, a list out."""
    out = []
    for at, bt in zip(a, b):
        h = torch.addcmul(bt, at, h)
        out.append(h)
    return out


def _gradients64(gate, x, h0, mix, dh, dhT):
    """Gradients of <h, dh> + <h_T, dhT> by the chain rule, token by token from the last."""
    a, w, slope = _mix64(gate, mix)
    states = _tokens64(a, w * x, h0)
    slope = slope * x + a * (1.0 / (1.0 + torch.exp(gate))) * torch.stack([h0, *states[:-1]])
    dx, dgate = torch.empty_like(x), torch.empty_like(gate)
    r = torch.zeros_like(h0) if dhT is None else dhT
    for t in range(x.shape[0] - 1, -1, -1):
        r = r + dh[t]
        torch.mul(w[t], r, out=dx[t])
        torch.mul(slope[t], r, out=dgate[t])
        r = a[t] * r
    return dx, dgate, r


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    wide = lambda x: None if x is None else x.double()  # noqa: E731
    if op in ("norm", "norm_train"):
        x, weight, bias = wide(s["x"]), wide(s["weight"]), wide(s["bias"])
        if op == "norm_train":
            x, weight, bias = (v.requires_grad_() for v in (x, weight, bias))
        total = x if s.get("residual") is None else x + wide(s["residual"])
        var, mean = torch.var_mean(total, dim=-1, keepdim=True, unbiased=False)
        y = (total - mean) / torch.sqrt(var + EPS) * weight + bias
        if op == "norm":
            return {"y": y} if s["residual"] is None else {"y": y, "s": total}
        loss = (y * wide(s["dy"])).sum()
        if s["ds"] is not None:
            loss = loss + (x * wide(s["ds"])).sum()
        return dict(zip(("x", "weight", "bias"), torch.autograd.grad(loss, (x, weight, bias))))
    if op == "step":
        a, w, _ = _mix64(wide(s["gate"]), case["mix"])
        h = a * wide(s["h"]) + w * wide(s["x"])
        return {"y": h, "h": h}
    B, C = case["B"], case["C"]
    first = lambda x: wide(x).transpose(0, 1).contiguous()  # noqa: E731
    gate, x = first(s["gate"]), first(s["x"])
    h0 = torch.zeros(B, C, dtype=torch.float64, device="cuda") if s["h0"] is None else wide(s["h0"])
    if op == "scan":
        a, w, _ = _mix64(gate, case["mix"])
        h = _tokens64(a, w * x, h0)
        return {"h": torch.stack(h, 1), "hT": h[-1]}
    dx, dgate, dh0 = _gradients64(gate, x, h0, case["mix"], first(s["dh"]), wide(s["dhT"]))
    out = {"x": dx.transpose(0, 1), "gate": dgate.transpose(0, 1)}
    if s["h0"] is not None:
        out["h0"] = dh0
    return out
