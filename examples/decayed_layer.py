"""The decayed linear-attention layer as a model uses it: a prompt, tokens one by one
from the state it leaves, and a training step.

    python -m preconditioned_delta_rule_phase1_gb300.build
    python examples/decayed_layer.py

The mixing is ``ops.decay_attn`` (``decay_attn_step`` for single tokens), its output
goes through ``ops.group_norm`` (a group a head, gated, channels last, which is what an
output projection reads), and the step ends with ``ops.clip_grad_norm``.  The
projections around them are plain matrix products.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from preconditioned_delta_rule_phase1_gb300 import ops  # noqa: E402

HEADS, K, V, WIDTH = 4, 64, 128, 256


class Layer:
    """x [B,T,WIDTH] -> [B,T,WIDTH], bf16; weights and gradients in dicts."""

    def __init__(self, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        new = lambda i, o: (torch.randn(i, o, generator=g, device=device) / i ** 0.5).bfloat16()  # noqa: E731
        self.w = {"q": new(WIDTH, HEADS * K), "k": new(WIDTH, HEADS * K), "v": new(WIDTH, HEADS * V),
                  "gate": new(WIDTH, HEADS * V), "out": new(HEADS * V, WIDTH),
                  "weight": torch.ones(HEADS * V, device=device),
                  "bias": torch.zeros(HEADS * V, device=device)}
        # memories from 32 to 4096 tokens
        self.decay = 1.0 - torch.exp2(-torch.linspace(5, 12, HEADS, device=device))
        self.ws = ops.Workspace(device=device)

    def _heads(self, x, name, width):
        y = (x @ self.w[name]).view(*x.shape[:2], HEADS, width)
        return y.transpose(1, 2).contiguous()

    def prompt(self, x, S0=None):
        """Returns (output, state, what the backward pass needs)."""
        q, k, v = (self._heads(x, n, w) for n, w in (("q", K), ("k", K), ("v", V)))
        o, ST = ops.decay_attn(q, k, v, self.decay, S0, workspace=self.ws)
        gate = x @ self.w["gate"]
        y = ops.group_norm(o, self.w["weight"], self.w["bias"], gate=gate, act="silu")
        return y @ self.w["out"], ST, (x, q, k, v, o, gate, y, S0)

    def token(self, x, S):
        """One token x [B,1,WIDTH], the state S updated in place."""
        q, k, v = (self._heads(x, n, w)[:, :, 0].contiguous() for n, w in (("q", K), ("k", K), ("v", V)))
        o = ops.decay_attn_step(q, k, v, self.decay, S, workspace=self.ws)
        y = ops.group_norm(o[:, :, None], self.w["weight"], self.w["bias"], gate=x @ self.w["gate"], act="silu")
        return y @ self.w["out"]

    def gradients(self, saved, dout):
        """Gradients of the weights given the cotangent of the layer's output."""
        x, q, k, v, o, gate, y, S0 = saved
        flat = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
        grads = {"out": flat(y).t() @ flat(dout)}
        n = ops.group_norm_backward(o, dout @ self.w["out"].t(), self.w["weight"], self.w["bias"], gate=gate,
                                    act="silu", workspace=self.ws)
        grads["weight"], grads["bias"] = n["weight"], n["bias"]
        grads["gate"] = flat(x).t() @ flat(n["gate"])
        a = ops.decay_attn_backward(q, k, v, self.decay, S0, do=n["x"], workspace=self.ws)
        for name in ("q", "k", "v"):
            grads[name] = flat(x).t() @ flat(a[name].transpose(1, 2).reshape(*x.shape[:2], -1))
        return grads


def main():
    torch.manual_seed(0)
    layer = Layer()
    x = torch.randn(2, 300, WIDTH, device="cuda").bfloat16()
    # a prompt of 297 tokens, then three tokens one by one, against the whole at once
    whole, _, saved = layer.prompt(x)
    part, S, _ = layer.prompt(x[:, :297].contiguous())
    tokens = [layer.token(x[:, t:t + 1].contiguous(), S) for t in range(297, 300)]
    off = (torch.cat([part, *tokens], 1).float() - whole.float()).abs().max() / whole.float().abs().max()
    # a training step towards a random target
    target = torch.randn_like(whole)
    loss = [float(((whole - target).float() ** 2).mean())]
    for _ in range(5):
        out, _, saved = layer.prompt(x)
        grads = layer.gradients(saved, ((out - target) * (2.0 / out.numel() * 1000)).contiguous())
        norm = ops.clip_grad_norm(grads.values(), 1.0, workspace=layer.ws)   # in place
        for name, g in grads.items():
            layer.w[name] -= (0.2 * g).to(layer.w[name].dtype)
        loss.append(float(((layer.prompt(x)[0] - target).float() ** 2).mean()))
    status = layer.ws.status()
    print("prompt and tokens against the whole: %.1e; loss %s; last gradient norm %.3f; status %d"
          % (off, " ".join("%.4f" % v for v in loss), float(norm), status))
    return float(off), loss, status


if __name__ == "__main__":
    main()
