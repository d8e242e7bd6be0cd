"""64-bit definitions of the layer operators for their tests (no code of the library).

Every function works on float64 tensors of any device.  `keep_mask` is the
published generator in Python integers over numpy words.
"""
import math

import numpy as np
import torch

MASK32 = 0xFFFFFFFF
UNIT = {torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11, torch.float32: 2.0**-24}  # half an ulp of 1
TINY = {torch.bfloat16: 2.0**-134, torch.float16: 2.0**-25, torch.float32: 2.0**-150}  # half the least subnormal


def philox(counter, key, rounds=7):
    """Philox4x32 of one counter (four words) under one key (two words), in Python integers."""
    c, k = list(counter), list(key)
    for _ in range(rounds):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & MASK32, (a >> 32) ^ c[3] ^ k[1], a & MASK32]
        k = [(k[0] + 0x9E3779B9) & MASK32, (k[1] + 0xBB67AE85) & MASK32]
    return c


def keep_mask(rows, cols, p, seed, offset):
    """(keep, scale): keep[row, col] by the definition in ozaki2_layers.h."""
    t = int(math.floor(65536 * p + 0.5))
    g = -(-cols // 8)
    c = [np.broadcast_to(np.arange(g, dtype=object), (rows, g)),
         np.broadcast_to(np.arange(rows, dtype=object)[:, None], (rows, g)), offset & MASK32, offset >> 32 & MASK32]
    words = philox(c, (seed & MASK32, seed >> 32 & MASK32))
    draws = np.stack([x for w in words for x in (np.broadcast_to(w, (rows, g)) % 65536, np.broadcast_to(w, (rows, g)) // 65536)], -1)
    keep = draws.reshape(rows, g * 8)[:, :cols].astype(np.int64) >= t
    return torch.from_numpy(keep), (65536.0 / (65536 - t) if t < 65536 else 0.0)


def act(z, name):
    if name == "none":
        return z
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return z * torch.special.ndtr(z)
    return z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z**3))) / 2


def slope(z, name):
    """act'(z), by autograd of the definition."""
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).double()
    z = z.detach().clone().requires_grad_(True)
    return torch.autograd.grad(act(z, name).sum(), z)[0]


def norm_rope(x, w, cos, sin, eps, interleaved):
    u = x * w / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    half = cos.shape[1]
    c, s = cos[:, None].double(), sin[:, None].double()
    if interleaved:
        a, b = u[..., 0:2 * half:2], u[..., 1:2 * half:2]
        v = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = u[..., :half], u[..., half:2 * half]
        v = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((v, u[..., 2 * half:]), -1)


def assert_within(got, want, bound, what=""):
    """Every element finite where it should be, and |got - want| <= bound."""
    got, want = got.double(), want.double()
    finite = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), finite), what
    assert torch.equal(got[~finite].nan_to_num(7.0), want[~finite].nan_to_num(7.0)), what
    over = ((got - want).abs() - bound)[finite]
    if over.numel():
        at = int(over.argmax())
        assert float(over.max()) <= 0, (what, float(got[finite][at]), float(want[finite][at]),
                                        float(bound.expand_as(want)[finite][at]) if torch.is_tensor(bound) else bound)
