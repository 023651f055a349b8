"""Cases of the decayed linear-attention layer: its attention (whole prompts, single
tokens, gradients), the group norm with an activation behind it, and the clipping of
a training step's gradients by their global norm.

Attention, per sequence (b, h), with the decay a = decay[h]:
    S_t = a S_{t-1} + v_t k_t^T,    o_t = S_t q_t        (S [V][K], fp32)
Group norm, per token and group of D channels, x^ = (x - mean) / sqrt(var + eps):
    z = weight x^ + bias,    y = act(z), or z act(gate) where a gate is given
Clipping, over all tensors g:
    n = sqrt(sum g^2),    g <- g max_norm / n where n > max_norm

``own`` false: the plain forms below, elementary torch operations in fp32.
``own`` true: the library's calls.
"""
import math
import random

import torch

own = False

CHUNK = 128          # tokens a chunk of the plain attention
EPS = 1e-5
MAX_NORM = 1.0
DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


# ----------------------------------------------------------------------- cases
def listed():
    return [
        # a short odd prompt in fp32, continued from a state: a parity run, or a user's first turn
        {"name": "prompt_odd_f32", "op": "prompt", "io": "f32", "B": 2, "H": 4, "T": 777,
         "K": 64, "V": 128, "S0": True},
        # the 340M-class layer over a batch of prompts
        {"name": "prompt_batch", "op": "prompt", "io": "bf16", "B": 8, "H": 8, "T": 2048,
         "K": 128, "V": 128, "S0": False},
        # one long document, read on from a state (the long-context layer)
        {"name": "prompt_long", "op": "prompt", "io": "bf16", "B": 1, "H": 16, "T": 65536,
         "K": 128, "V": 128, "S0": True},
        # one user's next token: latency
        {"name": "step_one", "op": "step", "io": "bf16", "B": 1, "H": 16, "K": 128, "V": 128},
        # a full serving batch's next token: the states' traffic
        {"name": "step_batch", "op": "step", "io": "bf16", "B": 256, "H": 16, "K": 128, "V": 128},
        # truncated back-propagation over an odd piece, with both states' gradients
        {"name": "train_odd", "op": "train", "io": "bf16", "B": 3, "H": 5, "T": 1037,
         "K": 128, "V": 64, "S0": True},
        # the 1.3B-class layer's training step
        {"name": "train_long", "op": "train", "io": "bf16", "B": 2, "H": 16, "T": 8192,
         "K": 128, "V": 128, "S0": False},
        # the norm behind step_batch
        {"name": "norm_token", "op": "norm", "io": "bf16", "B": 256, "H": 16, "T": 1, "D": 128,
         "heads_first": True, "gate": True, "act": "silu"},
        # the norm behind the 1.3B-class layer, from the attention's layout to channels last
        {"name": "norm_prompt", "op": "norm", "io": "bf16", "B": 2, "H": 16, "T": 8192, "D": 128,
         "heads_first": True, "gate": True, "act": "silu"},
        # its gradients, odd length, channels last on both sides
        {"name": "norm_train", "op": "norm_train", "io": "bf16", "B": 3, "H": 16, "T": 2731,
         "D": 128, "heads_first": False, "gate": True, "act": "silu"},
        # clipping a small model's gradients: latency
        {"name": "clip_small", "op": "clip", "tensors": 37, "elements": 1000003},
        # clipping a 340M-class model's gradients: bandwidth
        {"name": "clip_large", "op": "clip", "tensors": 266, "elements": 340000000},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "step", "train", "norm", "norm_train", "clip"])
    io = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("prompt", "train"):
        # token-heads bounded by the largest listed case of the op (a quarter of it in fp32)
        most = (1 << (20 if op == "prompt" else 18)) >> (2 if io == "f32" else 0)
        H = _log(rng, 1, 16)
        T = _log(rng, 1, min(65536, most // H))
        B = _log(rng, 1, max(1, min(8, most // (H * T))))
        return {"op": op, "io": io, "B": B, "H": H, "T": T, "K": rng.choice([64, 128]),
                "V": rng.choice([64, 128]), "S0": rng.random() < 0.5}
    if op == "step":
        return {"op": op, "io": io, "B": _log(rng, 1, 256), "H": _log(rng, 1, 16),
                "K": rng.choice([64, 128]), "V": rng.choice([64, 128])}
    if op == "clip":
        n = _log(rng, 1, 300)
        return {"op": op, "tensors": n, "elements": _log(rng, n, 200000000)}
    H, D = _log(rng, 1, 32), 8 * _log(rng, 1, 32)
    most = (1 << 25) // (H * D) >> (1 if io == "f32" else 0)
    T = _log(rng, 1, min(8192, most))
    B = _log(rng, 1, max(1, min(256, most // T)))
    return {"op": op, "io": io, "B": B, "H": H, "T": T, "D": D, "gate": rng.random() < 0.7,
            "heads_first": rng.random() < 0.5, "act": rng.choice(["none", "silu", "sigmoid"])}


def _sizes(case):
    """Element counts and types of the gradients: half small vectors in fp32, the rest
    matrices in bf16 whose sizes differ by up to 30 times."""
    rng = random.Random(case["tensors"] * 1000003 + case["elements"])
    n, total = case["tensors"], case["elements"]
    small = n // 2
    got = [(min(rng.randint(1, 4096), max(1, total // (4 * n))), torch.float32) for _ in range(small)]
    left = total - sum(s for s, _ in got)
    w = [math.exp(rng.uniform(0.0, 3.4)) for _ in range(n - small)]
    got += [(max(1, int(left * x / sum(w))), torch.bfloat16) for x in w]
    rng.shuffle(got)
    return got


def _views(sizes, fill):
    """One tensor a gradient, views of one buffer a type, each on a 256-byte boundary."""
    flat, at = {}, []
    for dt in (torch.float32, torch.bfloat16):
        off = 0
        for i, (n, d) in enumerate(sizes):
            if d == dt:
                at.append((i, dt, off, n))
                off += -(-n // 128) * 128
        flat[dt] = fill(off, dt)
    at.sort(key=lambda a: a[0])
    return flat, [flat[dt][off:off + n] for _, dt, off, n in at]


# ---------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    op = case["op"]
    s = {"case": case}
    if op == "clip":
        sizes = _sizes(case)
        flat, s["grads"] = _views(sizes, lambda n, dt: (normal(n) * 2e-3).to(dt))
        s["flat"], s["outs"] = _views(sizes, lambda n, dt: torch.zeros(n, dtype=dt, device="cuda"))
        return s
    B, H, dt = case["B"], case["H"], DTYPE[case["io"]]
    if op in ("norm", "norm_train"):
        T, D = case["T"], case["D"]
        s["x"] = (normal(*((B, H, T, D) if case["heads_first"] else (B, T, H * D))) * 0.4 + 0.1).to(dt)
        s["weight"], s["bias"] = 1.0 + 0.1 * normal(H * D), 0.1 * normal(H * D)
        s["gate"] = normal(B, T, H * D).to(dt) if case["gate"] else None
        if op == "norm_train":
            s["dy"] = normal(B, T, H * D).to(dt)
        return s
    K, V = case["K"], case["V"]
    T = () if op == "step" else (case["T"],)
    s["q"], s["k"] = (unit(normal(B, H, *T, K)).to(dt) for _ in range(2))
    s["v"] = normal(B, H, *T, V).to(dt)
    # memories from about 30 tokens to about 4000, one a head
    head = torch.arange(H, device="cuda") / max(1, H - 1)
    jitter = torch.rand(H, generator=g, device="cuda") * 0.5
    s["decay"] = 1.0 - torch.exp2(-(5.0 + 6.5 * head + jitter))
    if op == "step":
        s["S"] = normal(B, H, V, K)
    else:
        s["S0"] = normal(B, H, V, K) * 0.1 if case["S0"] else None
    if op == "train":
        s["do"] = normal(B, H, *T, V).to(dt)
        s["dST"] = normal(B, H, V, K) * 0.1 if case["S0"] else None
    return s


# ----------------------------------------------------------------- plain forms
def _chunks(x, n):
    x = x.float()
    B, H, T, W = x.shape
    pad = n * CHUNK - T
    if pad:
        x = torch.cat([x, x.new_zeros(B, H, pad, W)], 2)
    return x.reshape(B, H, n, CHUNK, W)


def _weights(decay, T):
    """Powers of the decay: within a chunk [H, 1, C, C], from a chunk's start [H, 1, C, 1],
    to its end [H, n, C, 1] (the last one may be short), between chunks [H, n, n]."""
    n = -(-T // CHUNK)
    a = decay.float()
    i = torch.arange(CHUNK, device=a.device)
    c = torch.arange(n, device=a.device)
    gap = i[:, None] - i[None, :]
    D = torch.where(gap >= 0, a[:, None, None] ** gap.clamp(min=0), 0.0)[:, None]
    first = (a[:, None] ** (i + 1))[:, None, :, None]
    length = (T - c * CHUNK).clamp(max=CHUNK)
    last = (a[:, None, None] ** (length[:, None] - 1 - i[None, :]).clamp(min=0))[..., None]
    gap = c[:, None] - 1 - c[None, :]
    across = torch.where(gap >= 0, a[:, None, None] ** (CHUNK * gap).clamp(min=0), 0.0)
    return n, D, first, last, across


def _starts(k, v, last, across, decay, S0):
    """The state entering each chunk [B, H, n, V, K], and what each chunk adds to it."""
    B, H, n, _, K = k.shape
    V = v.shape[-1]
    add = (v * last).transpose(-1, -2) @ k
    S = (across @ add.reshape(B, H, n, V * K)).reshape(B, H, n, V, K)
    if S0 is not None:
        c = torch.arange(n, device=k.device) * CHUNK
        S = S + (decay[:, None] ** c)[:, :, None, None] * S0[:, :, None]
    return S, add


def _prompt(s):
    T, a = s["q"].shape[2], s["decay"]
    n, D, first, last, across = _weights(a, T)
    q, k, v = (_chunks(s[x], n) for x in "qkv")
    S, add = _starts(k, v, last, across, a, s["S0"])
    o = ((q @ k.transpose(-1, -2)) * D) @ v + first * (q @ S.transpose(-1, -2))
    B, H = q.shape[:2]
    o = o.reshape(B, H, n * CHUNK, -1)[:, :, :T].to(s["q"].dtype)
    ST = (a ** (T - (n - 1) * CHUNK))[:, None, None] * S[:, :, -1] + add[:, :, -1]
    return {"o": o, "ST": ST}


def _train(s):
    T, a = s["q"].shape[2], s["decay"]
    n, D, first, last, across = _weights(a, T)
    q, k, v, do = (_chunks(s[x], n) for x in ("q", "k", "v", "do"))
    B, H, _, _, K = k.shape
    V = v.shape[-1]
    S, _ = _starts(k, v, last, across, a, s["S0"])
    # the cotangent of the state leaving each chunk
    add = (do * first).transpose(-1, -2) @ q
    G = (across.transpose(-1, -2) @ add.reshape(B, H, n, V * K)).reshape(B, H, n, V, K)
    c = torch.arange(n, device=k.device)
    dS0 = ((a[:, None] ** (CHUNK * c))[:, :, None, None] * add).sum(2)
    if s["dST"] is not None:
        left = (T - (c + 1) * CHUNK).clamp(min=0)
        G = G + (a[:, None] ** left)[:, :, None, None] * s["dST"][:, :, None]
        dS0 = dS0 + (a ** T)[:, None, None] * s["dST"]
    P = (q @ k.transpose(-1, -2)) * D
    dP = (do @ v.transpose(-1, -2)) * D
    dq = dP @ k + first * (do @ S)
    dk = dP.transpose(-1, -2) @ q + last * (v @ G)
    dv = P.transpose(-1, -2) @ do + last * (k @ G.transpose(-1, -2))
    out = {x: y.reshape(B, H, n * CHUNK, -1)[:, :, :T].to(s["q"].dtype)
           for x, y in (("q", dq), ("k", dk), ("v", dv))}
    if s["S0"] is not None:
        out["S0"] = dS0
    return out


def _step(s):
    S = s["S"]
    S.mul_(s["decay"][:, None, None]).add_(s["v"].float()[..., :, None] * s["k"].float()[..., None, :])
    o = (S * s["q"].float()[..., None, :]).sum(-1)
    return {"o": o.to(s["q"].dtype), "S": S}


def _act(z, act):
    return z if act == "none" else torch.sigmoid(z) if act == "sigmoid" else z * torch.sigmoid(z)


def _dact(z, act):
    if act == "none":
        return torch.ones_like(z)
    p = torch.sigmoid(z)
    return p * (1 - p) if act == "sigmoid" else p * (1 + z * (1 - p))


def _grouped(s, x):
    """[B, T, H, D] in fp32, from either layout."""
    c = s["case"]
    return x.float().transpose(1, 2) if c["heads_first"] else x.float().reshape(c["B"], c["T"], c["H"], c["D"])


def _norm(s):
    c = s["case"]
    x = _grouped(s, s["x"])
    m = x.mean(-1, keepdim=True)
    r = ((x - m).square().mean(-1, keepdim=True) + EPS).rsqrt()
    z = ((x - m) * r).reshape(c["B"], c["T"], -1) * s["weight"] + s["bias"]
    y = _act(z, c["act"]) if s["gate"] is None else z * _act(s["gate"].float(), c["act"])
    return y.to(s["x"].dtype)


def _norm_train(s):
    c = s["case"]
    x = _grouped(s, s["x"])
    m = x.mean(-1, keepdim=True)
    r = ((x - m).square().mean(-1, keepdim=True) + EPS).rsqrt()
    xh = (x - m) * r
    z = xh.reshape(c["B"], c["T"], -1) * s["weight"] + s["bias"]
    dy = s["dy"].float()
    out = {}
    if s["gate"] is None:
        dz = dy * _dact(z, c["act"])
    else:
        g = s["gate"].float()
        dz = dy * _act(g, c["act"])
        out["gate"] = (dy * z * _dact(g, c["act"])).to(s["x"].dtype)
    out["weight"] = (dz * xh.reshape(z.shape)).sum((0, 1))
    out["bias"] = dz.sum((0, 1))
    dh = (dz * s["weight"]).reshape(x.shape)
    dx = r * (dh - dh.mean(-1, keepdim=True) - xh * (dh * xh).mean(-1, keepdim=True))
    dx = dx.transpose(1, 2).contiguous() if c["heads_first"] else dx.reshape(z.shape)
    out["x"] = dx.to(s["x"].dtype)
    return out


def _clip(s):
    n = torch.stack([g.float().square().sum() for g in s["grads"]]).sum().sqrt()
    scale = torch.where(n > MAX_NORM, MAX_NORM / n, 1.0)
    [o.copy_(g.float() * scale) for g, o in zip(s["grads"], s["outs"])]
    return {"norm": n.reshape(1), "f32": s["flat"][torch.float32], "bf16": s["flat"][torch.bfloat16]}


PLAIN = {"prompt": _prompt, "step": _step, "train": _train, "norm": _norm,
         "norm_train": _norm_train, "clip": _clip}


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
    if op == "prompt":
        o, ST = ops.decay_attn(s["q"], s["k"], s["v"], s["decay"], s["S0"], workspace=ws)
        return {"o": o, "ST": ST}
    if op == "step":
        o = ops.decay_attn_step(s["q"], s["k"], s["v"], s["decay"], s["S"], workspace=ws)
        return {"o": o, "S": s["S"]}
    if op == "train":
        return ops.decay_attn_backward(s["q"], s["k"], s["v"], s["decay"], s["S0"], do=s["do"],
                                       dST=s["dST"], workspace=ws)
    if op == "clip":
        n = ops.clip_grad_norm(s["grads"], MAX_NORM, outs=s["outs"], workspace=ws)
        return {"norm": n, "f32": s["flat"][torch.float32], "bf16": s["flat"][torch.bfloat16]}
    if op == "norm":
        return ops.group_norm(s["x"], s["weight"], s["bias"], gate=s["gate"], groups=case["H"],
                              act=case["act"], eps=EPS)
    return ops.group_norm_backward(s["x"], s["dy"], s["weight"], s["bias"], gate=s["gate"],
                                   groups=case["H"], act=case["act"], eps=EPS, workspace=ws)


# ------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "clip":
        sizes = _sizes(case)
        n = sum(s for s, _ in sizes)
        return {"bytes": 2 * sum(s * (4 if d == torch.float32 else 2) for s, d in sizes) + 4, "flops": 3 * n}
    e = 4 if case["io"] == "f32" else 2
    B, H = case["B"], case["H"]
    if op in ("norm", "norm_train"):
        n, C = B * case["T"] * H * case["D"], H * case["D"]
        if op == "norm":
            return {"bytes": (3 if case["gate"] else 2) * n * e + 8 * C, "flops": 10 * n}
        return {"bytes": (5 if case["gate"] else 3) * n * e + 16 * C, "flops": 25 * n}
    K, V = case["K"], case["V"]
    if op == "step":
        return {"bytes": B * H * (8 * K * V + (2 * K + 2 * V) * e) + 4 * H, "flops": 5 * B * H * K * V}
    n, state = B * H * case["T"], 4 * B * H * K * V
    if op == "prompt":
        return {"bytes": n * (2 * K + 2 * V) * e + state * (2 if case["S0"] else 1) + 4 * H,
                "flops": 4 * n * K * V}
    # two states' updates and three products with them
    return {"bytes": n * (4 * K + 3 * V) * e + state * (3 if case["S0"] else 0) + 4 * H,
            "flops": 10 * n * K * V}


# ------------------------------------------------------------------------ 64 bits
def _attend64(q, k, v, a, S, block=256):
    """The recurrence block by block, carrying the state (autograd passes through)."""
    out = []
    for t in range(0, q.shape[2], block):
        qb, kb, vb = (x[:, :, t:t + block] for x in (q, k, v))
        L = qb.shape[2]
        i = torch.arange(L, device=q.device, dtype=torch.float64)
        lower = torch.tril(torch.ones(L, L, device=q.device, dtype=torch.float64))
        power = torch.exp((i[:, None] - i[None, :]) * lower * a.log()[:, None, None]) * lower
        near = ((qb @ kb.transpose(-1, -2)) * power) @ vb
        far = torch.einsum("bhik,bhvk->bhiv", qb, S) * (a[:, None] ** (i + 1))[None, :, :, None]
        out.append(near + far)
        S = S * (a ** L)[None, :, None, None] + \
            torch.einsum("bhjv,hj,bhjk->bhvk", vb, a[:, None] ** (L - 1 - i), kb)
    return torch.cat(out, 2), S


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    wide = lambda x: None if x is None else x.double()  # noqa: E731
    if op == "clip":
        n = math.sqrt(math.fsum(float(x.double().square().sum()) for x in s["grads"]))
        for x, o in zip(s["grads"], s["outs"]):
            o.copy_(x)
        c = min(1.0, MAX_NORM / n) if n > 0 else 1.0
        return {"norm": torch.tensor([n], dtype=torch.float64),
                "f32": s["flat"][torch.float32].double() * c,
                "bf16": s["flat"][torch.bfloat16].double() * c}
    if op in ("norm", "norm_train"):
        B, T, H, D = case["B"], case["T"], case["H"], case["D"]
        names = [x for x in ("x", "weight", "bias", "gate") if s[x] is not None]
        t = {x: wide(s[x]).requires_grad_(op == "norm_train") for x in names}
        x = t["x"].permute(0, 2, 1, 3) if case["heads_first"] else t["x"].view(B, T, H, D)
        var, mean = torch.var_mean(x, dim=-1, keepdim=True, unbiased=False)
        z = ((x - mean) / torch.sqrt(var + EPS)).reshape(B, T, H * D) * t["weight"] + t["bias"]
        u = t.get("gate", z)
        u = u if case["act"] == "none" else (u if case["act"] == "silu" else 1.0) / (1.0 + torch.exp(-u))
        y = z * u if "gate" in t else u
        if op == "norm":
            return y
        return dict(zip(names, torch.autograd.grad(y, [t[x] for x in names], wide(s["dy"]))))
    a = wide(s["decay"])
    if op == "step":
        S = a[:, None, None] * wide(s["S"]) + torch.einsum("bhv,bhk->bhvk", wide(s["v"]), wide(s["k"]))
        return {"o": torch.einsum("bhvk,bhk->bhv", S, wide(s["q"])), "S": S}
    train = op == "train"
    B, H, K, V = (case[x] for x in "BHKV")
    q, k, v = (wide(s[x]).requires_grad_(train) for x in "qkv")
    S0 = torch.zeros(B, H, V, K, dtype=torch.float64, device="cuda") if s["S0"] is None else wide(s["S0"])
    S0.requires_grad_(train)
    o, ST = _attend64(q, k, v, a, S0)
    if not train:
        return {"o": o, "ST": ST}
    loss = (o * wide(s["do"])).sum() + (0.0 if s["dST"] is None else (ST * wide(s["dST"])).sum())
    got = dict(zip(("q", "k", "v", "S0"), torch.autograd.grad(loss, (q, k, v, S0))))
    if s["S0"] is None:
        got.pop("S0")
    return got
