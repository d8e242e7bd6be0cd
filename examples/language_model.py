"""A small language model of norms, feed-forward pairs and a head, trained and asked for its next tokens.

    python examples/language_model.py

Everything but the embedding runs on the package's kernels: the norm in front
of each pair with the residual stream's addition in it, the products, the loss
with its gradient, and one AdamW step over all weights at once, 16-bit weights
beside 32-bit master copies and states in 32 or 8 bits.
"""
from __future__ import annotations

import importlib.util
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import emulated_fp64_gemm_gb300 as oz2  # noqa: E402

spec = importlib.util.spec_from_file_location("transformer_block", os.path.join(os.path.dirname(os.path.abspath(__file__)), "transformer_block.py"))
block = importlib.util.module_from_spec(spec)
spec.loader.exec_module(block)


class RmsNorm(torch.autograd.Function):
    """(norm of x + residual, x + residual), or of x alone where there is no residual."""

    @staticmethod
    def forward(ctx, x, weight, residual):
        y, s = oz2.rms_norm(x, weight, residual=residual) if residual is not None else (oz2.rms_norm(x, weight), x.view_as(x))
        ctx.save_for_backward(s, weight)
        ctx.residual = residual is not None
        return y, s

    @staticmethod
    def backward(ctx, dy, ds):
        s, weight = ctx.saved_tensors
        dx, dw = oz2.rms_norm_backward(dy, s, weight, dresidual=ds)
        return dx, dw, dx if ctx.residual else None


class TokenLogprobs(torch.autograd.Function):
    """(log p of the targets, entropy) of each row."""

    @staticmethod
    def forward(ctx, logits, targets):
        r = oz2.token_logprobs(logits, targets, entropy=True)
        ctx.save_for_backward(logits, targets, *r[:4])
        return r.logprobs, r.entropy

    @staticmethod
    def backward(ctx, dlogprobs, dentropy):
        logits, targets, *saved = ctx.saved_tensors
        return oz2.token_logprobs_backward(dlogprobs, logits, targets, oz2.TokenLogprobs(*saved, None, None), dentropy=dentropy), None


class Model:
    def __init__(self, vocab=2003, dim=512, hidden=2048, layers=2, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(n, k, scale):
            return (torch.randn(n, k, generator=g, device="cuda") * scale).to(dtype).requires_grad_(True)

        def vector(n, value):
            return torch.full((n,), value, dtype=dtype, device="cuda", requires_grad=True)

        self.layers = layers
        self.w = {"embed": weight(vocab, dim, 1.0), "norm": vector(dim, 1.0), "head": weight(vocab, dim, dim**-0.5)}
        for i in range(layers):
            self.w |= {f"norm{i}": vector(dim, 1.0), f"up{i}": weight(hidden, dim, dim**-0.5), f"up{i}_b": vector(hidden, 0.0),
                       f"down{i}": weight(dim, hidden, hidden**-0.5), f"down{i}_b": vector(dim, 0.0)}

    def logits(self, ids):
        w, plain = self.w, (0.0, 0, 0)
        s, h = w["embed"][ids], None
        for i in range(self.layers):
            y, s = RmsNorm.apply(s, w[f"norm{i}"], h)  # the stream, with the pair before it added
            up = block.Linear.apply(y, w[f"up{i}"], w[f"up{i}_b"], None, "silu", plain)
            h = block.Linear.apply(up, w[f"down{i}"], w[f"down{i}_b"], None, "none", plain)
        y, _ = RmsNorm.apply(h, w["norm"], s)
        return block.Linear.apply(y, w["head"], None, None, "none", plain)

    def loss_and_gradients(self, ids, targets, bonus=0.0):
        """Minus the mean log probability of the targets (those of -100 count nothing), less a bonus for entropy."""
        logprobs, entropy = TokenLogprobs.apply(self.logits(ids), targets)
        loss = -(logprobs.sum() + bonus * entropy.sum()) / len(ids)
        return loss.detach(), dict(zip(self.w, torch.autograd.grad(loss, list(self.w.values()))))

    def train(self, ids, targets, steps=8, bits=32, lr=2e-3):
        """Losses of a few AdamW steps."""
        params = list(self.w.values())
        state, losses = oz2.adamw_state(params, bits=bits, master=True), []
        for _ in range(steps):
            loss, grads = self.loss_and_gradients(ids, targets)
            oz2.adamw(params, list(grads.values()), state, lr=lr, weight_decay=0.01, seed=1)
            losses.append(loss)
        return [float(v) for v in losses]

    @torch.no_grad()
    def alternatives(self, ids, top=5):
        """(ids, log probabilities) of the most likely next tokens."""
        r = oz2.token_logprobs(self.logits(ids), torch.full_like(ids, -100), top=top)
        return r.top_ids, r.top_logprobs


def main():
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(0, 2003, (257,), generator=g, device="cuda")
    for bits in (32, 8):
        model = Model()
        losses = model.train(ids[:-1], ids[1:], bits=bits)
        print(f"training losses, states in {bits} bits:", " ".join(f"{v:.3f}" for v in losses))
    tokens, logprobs = model.alternatives(ids[:1])
    print("next token:", ", ".join(f"{t} ({v:.2f})" for t, v in zip(tokens[0].tolist(), logprobs[0].tolist())))


if __name__ == "__main__":
    main()
