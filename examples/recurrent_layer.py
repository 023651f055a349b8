"""The gated recurrent layer as a model uses it: blocks of norm, recurrence and output
along a residual stream; a prompt, tokens one by one from the states it leaves, and a
training step over a padded batch of two packed documents.

    python -m preconditioned_delta_rule_phase1_gb300.build
    python examples/recurrent_layer.py

Each block adds the previous block's output to the stream and norms the sum
(``ops.layer_norm`` with a residual), projects it to the recurrence's input and gate
(``ops.gated_scan``; ``gated_scan_step`` for single tokens) and projects its state to the
output.  The step ends with ``ops.clip_grad_norm``.  The projections are plain matrix
products.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from preconditioned_delta_rule_phase1_gb300 import ops  # noqa: E402

WIDTH, CHANNELS, BLOCKS = 256, 320, 2


class Model:
    """x [B,T,WIDTH] -> [B,T,WIDTH], bf16; weights and gradients in lists of dicts."""

    def __init__(self, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        new = lambda i, o: (torch.randn(i, o, generator=g, device=device) / i ** 0.5).bfloat16()  # noqa: E731
        self.w = [{"x": new(WIDTH, CHANNELS), "gate": new(WIDTH, CHANNELS), "out": new(CHANNELS, WIDTH),
                   # memories from 3 tokens to 1000, before the token moves them
                   "memory": torch.linspace(1, 7, CHANNELS, device=device).bfloat16(),
                   "weight": torch.ones(WIDTH, device=device), "bias": torch.zeros(WIDTH, device=device)}
                  for _ in range(BLOCKS)]
        self.ws = ops.Workspace(device=device)

    def gates(self, w, y, first=None, padded=None):
        """The gate's logits; documents start and padding passes by what it is set to."""
        gate = y @ w["gate"] + w["memory"]
        if first is not None:
            gate = gate.masked_fill(first[..., None], -math.inf)
        if padded is not None:
            gate = gate.masked_fill(padded[..., None], math.inf)
        return gate

    def prompt(self, x, states=None, first=None, padded=None):
        """Returns (output, states, what the backward pass needs)."""
        saved, ends, out = [], [], None
        for i, w in enumerate(self.w):
            if out is None:
                y, s = ops.layer_norm(x, w["weight"], w["bias"]), x
            else:
                y, s = ops.layer_norm(out, w["weight"], w["bias"], residual=s)
            xs, gate = y @ w["x"], self.gates(w, y, first, padded)
            h0 = None if states is None else states[i]
            h, hT = ops.gated_scan(xs, gate, h0, mix="unit")
            out = h @ w["out"]
            ends.append(hT)
            saved.append((s, y, xs, gate, h, h0))
        return s + out, ends, saved

    def token(self, x, states):
        """One token x [B,WIDTH], the states updated in place."""
        out = None
        for w, state in zip(self.w, states):
            if out is None:
                y, s = ops.layer_norm(x, w["weight"], w["bias"]), x
            else:
                y, s = ops.layer_norm(out, w["weight"], w["bias"], residual=s)
            out = ops.gated_scan_step(y @ w["x"], self.gates(w, y), state, mix="unit") @ w["out"]
        return s + out

    def gradients(self, saved, dout):
        """Gradients of the weights, and of x, given the cotangent of the output."""
        flat = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
        grads, ds = [], dout        # of the stream, which every block's output is added to
        for w, (s, y, xs, gate, h, h0) in zip(reversed(self.w), reversed(saved)):
            g = {"out": flat(h).t() @ flat(ds)}
            a = ops.gated_scan_backward(xs, gate, h, h0, dh=ds @ w["out"].t(), mix="unit")
            g["x"], g["gate"] = flat(y).t() @ flat(a["x"]), flat(y).t() @ flat(a["gate"])
            g["memory"] = flat(a["gate"]).float().sum(0).bfloat16()
            n = ops.layer_norm_backward(s, a["x"] @ w["x"].t() + a["gate"] @ w["gate"].t(), w["weight"], w["bias"],
                                        ds=ds, workspace=self.ws)
            g["weight"], g["bias"], ds = n["weight"], n["bias"], n["x"]
            grads.insert(0, g)
        return grads, ds


def main():
    torch.manual_seed(0)
    model = Model()
    x = torch.randn(2, 300, WIDTH, device="cuda").bfloat16()
    # a prompt of 297 tokens, then three tokens one by one, against the whole at once
    whole, _, _ = model.prompt(x)
    part, states, _ = model.prompt(x[:, :297].contiguous())
    tokens = [model.token(x[:, t].contiguous(), states)[:, None] for t in range(297, 300)]
    off = (torch.cat([part, *tokens], 1).float() - whole.float()).abs().max() / whole.float().abs().max()
    # a second document from token 130 on, the second sequence padded from token 250 on
    first, padded = (torch.zeros(2, 300, dtype=torch.bool, device="cuda") for _ in range(2))
    first[:, 130], padded[1, 250:] = True, True
    target = torch.randn_like(whole)
    loss = []
    for _ in range(6):
        out, ends, saved = model.prompt(x, first=first, padded=padded)
        err = (out - target).masked_fill(padded[..., None], 0)
        loss.append(float((err.float() ** 2).mean()))
        grads, _ = model.gradients(saved, (err * (2.0 / out.numel() * 1000)).contiguous())
        norm = ops.clip_grad_norm([g for b in grads for g in b.values()], 1.0, workspace=model.ws)   # in place
        for w, g in zip(model.w, grads):
            for name in g:
                w[name] -= (0.2 * g[name]).to(w[name].dtype)
    status = model.ws.status()
    print("prompt and tokens against the whole: %.1e; loss %s; last gradient norm %.3f; status %d"
          % (off, " ".join("%.4f" % v for v in loss), float(norm), status))
    return float(off), loss, status


if __name__ == "__main__":
    main()
