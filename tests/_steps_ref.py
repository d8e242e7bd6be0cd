"""Definitions of the step operators for their tests: 64 bits, and single roundings in numpy for the 8-bit states
(no code of the library)."""
import numpy as np
import torch

from tests._layers_ref import MASK32, philox

F32 = np.float32


def rms_norm(x, w, residual, eps):
    s = x if residual is None else x + residual
    return s / torch.sqrt((s * s).sum(-1, keepdim=True) / s.shape[1] + eps) * w, s


def rms_norm_backward(dy, x, w, dres, eps):
    """(dx, dweight, and for each element the sum of the magnitudes that dx is the difference of)."""
    n = x.shape[1]
    r = 1 / torch.sqrt((x * x).sum(-1, keepdim=True) / n + eps)
    g = dy * w
    mean = (g * x).sum(-1, keepdim=True) / n
    dx = r * (g - x * r * r * mean)
    size = r * (g.abs() + x.abs() * r * r * (g * x).abs().sum(-1, keepdim=True) / n)
    if dres is not None:
        dx, size = dx + dres, size + dres.abs()
    return dx, (dy * x * r).sum(0), size, (dy * x * r).abs().sum(0)


def token_logprobs(logits, targets, temperature, ignore):
    """z_max, log_sum, the targets' log p, entropy and all log p of rows that have a distribution, or -inf alone."""
    # z below the 32-bit range is masked, like -inf: the lowest logits there are over a temperature below 1 (max / 0.7 > max)
    z = logits.double() / temperature
    z = torch.where(z < -torch.finfo(torch.float32).max, -np.inf, z)
    z_max = z.amax(-1)
    some = z_max > -np.inf
    d = z - torch.where(some, z_max, 0.0)[:, None]
    log_sum = torch.where(some, torch.log(torch.exp(d).sum(-1)), 0.0)
    logp = d - log_sum[:, None]
    p = torch.exp(logp)
    entropy = -torch.where(p > 0, p * logp, 0.0).sum(-1)
    inside = (targets >= 0) & (targets < logits.shape[1])
    t = torch.where(inside, logp.gather(1, torch.where(inside, targets, 0)[:, None])[:, 0], np.nan)
    return z_max, log_sum, torch.where(targets == ignore, 0.0, t), entropy, logp


def e4m3_values():
    """The values of the 256 codes: sign, four bits of exponent (bias 7), three of fraction; no infinity."""
    out = np.empty(256, np.float64)
    for c in range(256):
        e, f = c >> 3 & 15, c & 7
        v = f * 2.0**-9 if e == 0 else (8 + f) * 2.0**(e - 10)
        if c & 127 == 127:
            v = np.nan
        out[c] = -v if c >> 7 else v
    return out


E4M3 = e4m3_values()


def to_e4m3(x):
    """Codes of float32 values, to nearest, ties to even fractions, past the largest the largest."""
    grid = E4M3[:127]
    a = np.minimum(np.abs(x.astype(np.float64)), 448.0)
    hi = np.searchsorted(grid, a).clip(1, 126)
    lo = hi - 1
    up = a - grid[lo] > grid[hi] - a
    tie = a - grid[lo] == grid[hi] - a
    code = np.where(up | (tie & (hi % 2 == 0)), hi, lo).astype(np.uint8)
    return np.where(np.signbit(x), code | 128, code).astype(np.uint8)


def fourth(k):
    k = k.astype(F32)
    return (k * k) * (k * k)


def draws(groups, step, seed):
    """The eight 16-bit draws of each group of eight elements."""
    g = np.asarray(groups, dtype=object)
    words = philox([g % 2**32, g // 2**32, step & MASK32, step >> 32], (seed & MASK32, seed >> 32 & MASK32))
    cols = [x for w in words for x in (np.broadcast_to(w, g.shape) % 65536, np.broadcast_to(w, g.shape) // 65536)]
    return np.stack(cols, -1).astype(np.int64).reshape(-1)


def adamw_moments8(m_code, v_code, m_scale, v_scale, g, beta1, beta2, step, seed, first_group):
    """One step of a tensor's 8-bit states in single roundings: (m, v, their codes and scales); sizes multiples of 256,
    with zeros past the tensor's end."""
    blocks = g.size // 256
    spread = lambda s: np.repeat(s.astype(F32), 256)  # noqa: E731
    m = E4M3[m_code].astype(F32) * spread(m_scale)
    v = fourth(v_code) * spread(v_scale)
    m = F32(beta1) * m + F32(1.0 - beta1) * g
    v = F32(beta2) * v + F32(1.0 - beta2) * (g * g)
    top = lambda a: np.abs(a).reshape(blocks, 256).max(1)  # noqa: E731
    ms = np.maximum(top(m) * F32(1.0 / 448.0), F32(1e-36))
    vs = np.maximum(top(v) * F32(255.0**-4), F32(1e-36))
    mq = to_e4m3(m * spread(F32(1) / ms))
    t = v * spread(F32(1) / vs)
    ladder = fourth(np.arange(256))
    k = np.searchsorted(ladder, t, side="right") - 1
    low, high = ladder[k], fourth(k + 1)
    d = draws(np.arange(g.size // 8) + first_group, step, seed)
    up = ((t - low) * F32(65536) > d.astype(F32) * (high - low)) | ((k == 0) & (t > 0))
    return m, v, mq, np.minimum(k + up, 255).astype(np.uint8), ms, vs
