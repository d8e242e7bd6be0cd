"""One transformer block on the layer operators: a few training steps, then single tokens.

    python examples/transformer_block.py

The dense parts run on the package's kernels: the joined QKV projection, the
norm and rotation of queries and keys, the output projection with dropout and
residual, and the feed-forward pair.  Attention itself is left to plain torch.
The autograd functions below show which outputs a backward pass needs to keep:
no mask, and of an activation only its input.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import emulated_fp64_gemm_gb300 as oz2  # noqa: E402


class Linear(torch.autograd.Function):
    """residual + dropout(activation(x w^T + b)); a dropout's (p, seed, offset) stands for its mask."""

    @staticmethod
    def forward(ctx, x, w, b, residual, activation, drop):
        p, seed, offset = drop
        save = activation != "none"
        out = oz2.linear(x, w, b, activation=activation, residual=residual, dropout=p, seed=seed, offset=offset, save_preact=save)
        y, z = out if save else (out, None)
        ctx.save_for_backward(x, w, z)
        ctx.rest = activation, drop, residual is not None
        return y

    @staticmethod
    def backward(ctx, dy):
        x, w, z = ctx.saved_tensors
        activation, (p, seed, offset), residual = ctx.rest
        dx, dw, db = oz2.linear_backward(dy, x, w, preact=z, activation=activation, dropout=p, seed=seed, offset=offset,
                                         need_dx=ctx.needs_input_grad[0])
        return dx, dw, db, dy if residual else None, None, None


class Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, p, seed, offset):
        ctx.rest = p, seed, offset
        return oz2.dropout(x, p, seed=seed, offset=offset)

    @staticmethod
    def backward(ctx, dy):
        p, seed, offset = ctx.rest
        return oz2.dropout_backward(dy, p, seed=seed, offset=offset), None, None, None


class QkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, wq, wk, cos, sin, positions):
        ctx.save_for_backward(q, k, wq, wk, cos, sin, positions)
        return oz2.qk_norm_rope(q, k, wq, wk, cos, sin, positions)

    @staticmethod
    def backward(ctx, dq, dk):
        return (*oz2.qk_norm_rope_backward(dq, dk, *ctx.saved_tensors), None, None, None)


class Block:
    def __init__(self, dim=512, heads=8, kv_heads=2, head_dim=64, hidden=2048, context=1024, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(n, k):
            return (torch.randn(n, k, generator=g, device="cuda") * k**-0.5).to(dtype).requires_grad_(True)

        def vector(n, value):
            return torch.full((n,), value, dtype=dtype, device="cuda", requires_grad=True)

        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        joined = (heads + 2 * kv_heads) * head_dim
        self.w = {"qkv": weight(joined, dim), "qkv_b": vector(joined, 0.0), "wq": vector(head_dim, 1.0), "wk": vector(head_dim, 1.0),
                  "out": weight(dim, heads * head_dim), "out_b": vector(dim, 0.0), "up": weight(hidden, dim), "up_b": vector(hidden, 0.0),
                  "down": weight(dim, hidden), "down_b": vector(dim, 0.0)}
        angle = torch.arange(context, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(0, head_dim, 2, device="cuda", dtype=torch.float64) / head_dim)
        self.cos, self.sin = angle.cos().float(), angle.sin().float()

    def attention(self, q, k, v, mask):
        """softmax(q k^T / sqrt(d) + mask) v by torch; q (tokens, heads, d), k and v (past, kv_heads, d)."""
        group = self.heads // self.kv_heads
        k, v = (t.float().repeat_interleave(group, 1) for t in (k, v))
        scores = torch.einsum("thd,shd->hts", q.float(), k) * self.head_dim**-0.5 + mask
        return torch.einsum("hts,shd->thd", scores.softmax(-1), v).to(q.dtype).flatten(1)

    def __call__(self, x, positions, p=0.0, seed=0, step=0, cache=None):
        """x (tokens, dim).  With `cache` (a list of past keys and values) the tokens follow those of the cache."""
        w, h, kv, d = self.w, self.heads, self.kv_heads, self.head_dim
        drops = [(p, seed, 4 * step + i) for i in range(3)]  # an offset for each dropout of each step
        x = Dropout.apply(x, *drops[0])
        qkv = Linear.apply(x, w["qkv"], w["qkv_b"], None, "none", (0.0, 0, 0)).view(-1, h + 2 * kv, d)
        q, k = QkNormRope.apply(qkv[:, :h], qkv[:, h:h + kv], w["wq"], w["wk"], self.cos, self.sin, positions)
        v = qkv[:, h + kv:]
        if cache is not None:
            cache.append((k, v))
            k, v = (torch.cat(t) for t in zip(*cache))
        seen = torch.arange(k.shape[0], device="cuda")[None] <= positions[:, None]
        mask = torch.zeros(seen.shape, device="cuda").masked_fill_(~seen, float("-inf"))
        x = Linear.apply(self.attention(q, k, v, mask), w["out"], w["out_b"], x, "none", drops[1])
        up = Linear.apply(x, w["up"], w["up_b"], None, "gelu_tanh", (0.0, 0, 0))
        return Linear.apply(up, w["down"], w["down_b"], x, "none", drops[2])


def train(block, tokens=256, steps=8, rate=0.2, p=0.1):
    """Losses of a few steps of gradient descent towards a fixed output."""
    g = torch.Generator(device="cuda").manual_seed(1)
    dim = block.w["out_b"].numel()
    x = torch.randn(tokens, dim, generator=g, device="cuda").to(block.w["qkv"].dtype)
    target = torch.randn(tokens, dim, generator=g, device="cuda")
    positions = torch.arange(tokens, device="cuda")
    losses = []
    for step in range(steps):
        loss = (block(x, positions, p, seed=7, step=step).float() - target).square().mean()
        grads = torch.autograd.grad(loss, list(block.w.values()))
        with torch.no_grad():
            for value, grad in zip(block.w.values(), grads):
                value -= rate * grad
        losses.append(loss.detach())
    return [float(v) for v in losses]


@torch.no_grad()
def decode(block, x):
    """The block's outputs for the rows of x, one token at a time over a growing cache."""
    cache = []
    return torch.cat([block(x[i:i + 1], torch.tensor([i], device="cuda"), cache=cache) for i in range(x.shape[0])])


def main():
    block = Block()
    losses = train(block)
    print("training losses:", " ".join(f"{v:.3f}" for v in losses))
    x = torch.randn(32, 512, device="cuda").to(torch.bfloat16)
    with torch.no_grad():
        whole = block(x, torch.arange(32, device="cuda"))
    single = decode(block, x)
    print(f"one token at a time against the whole prompt: {float((whole - single).abs().max() / whole.abs().max()):.4f} of the largest output")


if __name__ == "__main__":
    main()
