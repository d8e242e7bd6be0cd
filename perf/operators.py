"""Measured cases of the layer operators: linear, linear_backward, dropout and qk_norm_rope.

Each case is one pass through one operator of a transformer block's dense part.
With `own` false, `run` computes it in elementary torch operations in 32 bits,
rounded once at the end; with `own` true it calls the package's operator.
`exact` computes it in 64 bits, by other formulas where there are any.

Definitions that both sides share:

* linear: z = x w^T + b, y = residual + keep * act(z) / (1 - p), z returned too where it is saved;
* linear_backward: dz = act'(z) * keep * dy / (1 - p), dx = dz w, dw = dz^T x, db = column sums of dz;
* dropout: y = residual + keep * x / (1 - p), and the same mask on the gradient;
* keep(row, col): Philox4x32 with 7 rounds (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy
  as 1, 2, 3", SC 2011), counter (col // 8, row, offset low, offset high), key (seed low, seed high); its four
  words give eight 16-bit draws for eight neighbouring columns, low half first; an element stays where its
  draw is at least T = round(65536 p), and p in the scale above stands for T / 65536;
* qk_norm_rope: per token and head, u = x w / sqrt(mean(x^2) + eps), then the first `rot` features are rotated
  by the token's position, in pairs (i, i + rot / 2) or, interleaved, (2 i, 2 i + 1).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32}
EPS = 1e-6
POSITIONS = 32768  # rows of the rotation tables
GELU_C, GELU_A = math.sqrt(2.0 / math.pi), 0.044715


# ------------------------------------------------------------------ cases
def _linear(m, k, n, dtype, act, bias=True, residual=False, p=0.0, save=False):
    return {"op": "linear", "m": m, "k": k, "n": n, "dtype": dtype, "act": act, "bias": bias, "residual": residual,
            "p": p, "save": save}


def _linear_backward(m, k, n, dtype, act, p=0.0):
    return {"op": "linear_backward", "m": m, "k": k, "n": n, "dtype": dtype, "act": act, "p": p}


def _dropout(m, n, dtype, p, residual=False, backward=False):
    return {"op": "dropout", "m": m, "n": n, "dtype": dtype, "p": p, "residual": residual, "backward": backward}


def _qk(t, hq, hkv, d, rot, dtype, interleaved=False, backward=False):
    return {"op": "qk_norm_rope", "t": t, "hq": hq, "hkv": hkv, "d": d, "rot": rot, "dtype": dtype,
            "interleaved": interleaved, "backward": backward}


def listed():
    return [
        # one new token through a small layer: launch latency
        dict(_linear(1, 1024, 4096, "bfloat16", "silu"), name="linear, one token"),
        # a serving batch of single tokens: reading the weights once
        dict(_linear(24, 8192, 8192, "bfloat16", "none", residual=True), name="linear, serving batch"),
        # nothing is a multiple of anything: a pruned or concatenated layer
        dict(_linear(333, 1999, 2051, "float16", "gelu", residual=True, p=0.1), name="linear, ragged"),
        # the first product of a feed-forward pair in training: the pre-activation is kept for the backward pass
        dict(_linear(8192, 4096, 16384, "bfloat16", "gelu_tanh", save=True), name="linear, up, training"),
        # the second one, with the block's dropout and residual
        dict(_linear(8192, 8192, 2048, "bfloat16", "none", residual=True, p=0.1), name="linear, down, dropout"),
        # the first product's backward pass
        dict(_linear_backward(8192, 4096, 16384, "bfloat16", "gelu_tanh"), name="linear backward, up"),
        # a fine-tuning micro-batch of odd length, with dropout after the activation
        dict(_linear_backward(517, 1024, 1531, "float16", "silu", p=0.2), name="linear backward, ragged"),
        # dropout on a small batch: latency
        dict(_dropout(64, 1000, "float16", 0.1, residual=True), name="dropout, small"),
        # the gradient through the residual branch's dropout of a long batch
        dict(_dropout(16384, 8192, "bfloat16", 0.1, backward=True), name="dropout backward, large"),
        # queries and keys of a serving batch
        dict(_qk(24, 32, 8, 128, 128, "bfloat16"), name="qk_norm_rope, serving batch"),
        # queries and keys of a prompt or a training batch
        dict(_qk(8192, 32, 8, 128, 128, "bfloat16"), name="qk_norm_rope, prompt"),
        # their gradients, with a partial, interleaved rotation in 32 bits
        dict(_qk(4096, 16, 4, 96, 64, "float32", interleaved=True, backward=True), name="qk_norm_rope backward"),
    ]


def _size(rng, low, high):
    """A size spread over the logarithm of the range: a multiple of 64, of 8, or any."""
    v = int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))
    step = rng.choice((64, 64, 8, 1))
    if v > step:
        v -= v % step
    v = max(low, min(high, v))
    return 3080 if v == 3072 else v


def draw(rng):
    op = rng.choice(("linear", "linear", "linear_backward", "dropout", "qk_norm_rope"))
    half = rng.choice(("bfloat16", "float16"))
    if op == "dropout":
        return _dropout(_size(rng, 1, 16384), _size(rng, 64, 8192), rng.choice((half, half, "float32")),
                        rng.choice((0.0, 0.1, 0.25, 0.5)), rng.random() < 0.5, rng.random() < 0.5)
    if op == "qk_norm_rope":
        d = rng.choice((64, 80, 96, 128, 128, 256, 2 * rng.randint(16, 128)))
        rot = rng.choice((d, d, d // 2 // 2 * 2))
        hkv = rng.choice((1, 2, 4, 8))
        return _qk(_size(rng, 1, 8192), hkv * rng.choice((1, 3, 4)), hkv, d, rot, rng.choice((half, half, "float32")),
                   rng.random() < 0.3, rng.random() < 0.5)
    while True:
        m, k, n = _size(rng, 1, 8192), _size(rng, 64, 8192), _size(rng, 64, 16384)
        if m * k * n <= 8192 * 4096 * 16384 // 2:
            break
    act, p = rng.choice(("none", "relu", "silu", "gelu", "gelu_tanh")), rng.choice((0.0, 0.0, 0.1, 0.3))
    if op == "linear_backward":
        return _linear_backward(m, k, n, half, act, p)
    return _linear(m, k, n, half, act, rng.random() < 0.8, rng.random() < 0.5, p, rng.random() < 0.3)


def work(case):
    size = torch.empty(0, dtype=DTYPES[case["dtype"]]).element_size()
    if case["op"] in ("linear", "linear_backward"):
        m, k, n = case["m"], case["k"], case["n"]
        if case["op"] == "linear":
            elements = m * k + n * k + m * n * (1 + case["residual"] + case["save"]) + n * case["bias"]
            return {"bytes": size * elements, "flops": 2.0 * m * k * n}
        elements = 2 * (m * k + n * k) + m * n * (1 + (case["act"] != "none")) + n
        return {"bytes": size * elements, "flops": 4.0 * m * k * n}
    if case["op"] == "dropout":
        return {"bytes": size * case["m"] * case["n"] * (2 + (case["residual"] and not case["backward"])), "flops": 0.0}
    heads = case["t"] * (case["hq"] + case["hkv"])
    tables = case["t"] * (4 * case["rot"] + 8) + 2 * case["d"] * size
    if case["backward"]:
        return {"bytes": 3 * size * heads * case["d"] + tables + 2 * case["d"] * size, "flops": 0.0}
    return {"bytes": 2 * size * heads * case["d"] + tables, "flops": 0.0}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(scale).to(dtype)

    s = dict(case, seed=(seed * 0x9E3779B97F4A7C15 + 1) % 2**63, offset=seed % 1000)
    if case["op"] in ("linear", "linear_backward"):
        m, k, n = case["m"], case["k"], case["n"]
        s["x"], s["w"] = normal(m, k), normal(n, k, scale=k**-0.5)
        if case["op"] == "linear":
            s["b"] = normal(n, scale=0.2) if case["bias"] else None
            s["res"] = normal(m, n) if case["residual"] else None
        else:
            s["dy"] = normal(m, n)
            s["z"] = normal(m, n) if case["act"] != "none" else None
    elif case["op"] == "dropout":
        s["x"] = normal(case["m"], case["n"])
        s["res"] = normal(case["m"], case["n"]) if case["residual"] and not case["backward"] else None
    else:
        t, hq, hkv, d, rot = case["t"], case["hq"], case["hkv"], case["d"], case["rot"]
        qkv = normal(t, hq + 2 * hkv, d)  # the product of the joined projection; the values are left alone
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv]
        s["wq"], s["wk"] = ((1.0 + 0.1 * normal(d).float()).to(dtype) for _ in range(2))
        angle = torch.arange(POSITIONS, device="cuda", dtype=torch.float64)[:, None] * torch.exp(
            torch.arange(rot // 2, device="cuda", dtype=torch.float64) * (-2.0 * math.log(10000.0) / rot))
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        s["pos"] = torch.randint(0, POSITIONS, (t,), generator=g, device="cuda")
        if case["backward"]:
            s["dq"], s["dk"] = normal(t, hq, d), normal(t, hkv, d)
    return s


# ------------------------------------------------------------------ plain forms
def _keep(rows, cols, p, seed, offset):
    """The mask and its scale, in whole-number torch operations."""
    mask32 = 0xFFFFFFFF
    groups = -(-cols // 8)
    c0 = torch.arange(groups, device="cuda").expand(rows, groups)
    c1 = torch.arange(rows, device="cuda")[:, None].expand(rows, groups)
    c2, c3 = torch.full_like(c0, offset & mask32), torch.full_like(c0, offset >> 32 & mask32)
    k0, k1 = seed & mask32, seed >> 32 & mask32
    for _ in range(7):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (b >> 32 & mask32) ^ c1 ^ k0, b & mask32, (a >> 32 & mask32) ^ c3 ^ k1, a & mask32
        k0, k1 = (k0 + 0x9E3779B9) & mask32, (k1 + 0xBB67AE85) & mask32
    words = torch.stack((c0, c0 >> 16, c1, c1 >> 16, c2, c2 >> 16, c3, c3 >> 16), -1) & 0xFFFF
    t = round(65536 * p)
    return words.reshape(rows, groups * 8)[:, :cols] >= t, 65536.0 / (65536 - t)


def _drop(v, p, seed, offset):
    if round(65536 * p) == 0:
        return v
    keep, scale = _keep(v.shape[0], v.shape[1], p, seed, offset)
    return torch.where(keep, v * scale, 0.0)


def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return z * (z > 0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return z * 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
    return z / (1 + torch.exp(-2 * GELU_C * (z + GELU_A * z * z * z)))


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s + z * s * (1 - s)
    s = 1 / (1 + torch.exp(-2 * GELU_C * (z + GELU_A * z * z * z)))
    return s + z * s * (1 - s) * (2 * GELU_C * (1 + 3 * GELU_A * z * z))


def _linear_plain(s):
    dtype = s["x"].dtype
    z = s["x"].float() @ s["w"].float().t()
    if s["b"] is not None:
        z += s["b"].float()
    y = _drop(_act(z, s["act"]), s["p"], s["seed"], s["offset"])
    if s["res"] is not None:
        y = y + s["res"].float()
    return {"y": y.to(dtype), "z": z.to(dtype)} if s["save"] else {"y": y.to(dtype)}


def _linear_backward_plain(s):
    dtype = s["x"].dtype
    dz = _drop(s["dy"].float(), s["p"], s["seed"], s["offset"])
    if s["z"] is not None:
        dz = dz * _act_slope(s["z"].float(), s["act"])
    return {"dx": (dz @ s["w"].float()).to(dtype), "dw": (dz.t() @ s["x"].float()).to(dtype), "db": dz.sum(0).to(dtype)}


def _dropout_plain(s):
    y = _drop(s["x"].float(), s["p"], s["seed"], s["offset"])
    return (y if s["res"] is None else y + s["res"].float()).to(s["x"].dtype)


def _turn(u, cos, sin, interleaved):
    half = cos.shape[1]
    c, s = cos[:, None], sin[:, None]
    if interleaved:
        a, b = u[..., 0:2 * half:2], u[..., 1:2 * half:2]
        turned = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = u[..., :half], u[..., half:2 * half]
        turned = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((turned, u[..., 2 * half:]), -1)


def _norm_rope_plain(x, w, cos, sin, interleaved):
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return _turn(x * r * w.float(), cos, sin, interleaved).to(w.dtype)


def _norm_rope_backward_plain(dy, x, w, cos, sin, interleaved):
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    g = _turn(dy.float(), cos, -sin, interleaved)
    gw = g * w.float()
    dx = r * (gw - x * (r * r * (gw * x).mean(-1, keepdim=True)))
    return dx.to(w.dtype), (g * x * r).sum((0, 1)).to(w.dtype)


def _qk_plain(s):
    cos, sin = s["cos"][s["pos"]], s["sin"][s["pos"]]
    if not s["backward"]:
        return {"q": _norm_rope_plain(s["q"], s["wq"], cos, sin, s["interleaved"]),
                "k": _norm_rope_plain(s["k"], s["wk"], cos, sin, s["interleaved"])}
    dq, dwq = _norm_rope_backward_plain(s["dq"], s["q"], s["wq"], cos, sin, s["interleaved"])
    dk, dwk = _norm_rope_backward_plain(s["dk"], s["k"], s["wk"], cos, sin, s["interleaved"])
    return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


# ------------------------------------------------------------------ the package's operators
def _run_own(s):
    import emulated_fp64_gemm_gb300 as oz2

    if s["op"] == "linear":
        y = oz2.linear(s["x"], s["w"], s["b"], activation=s["act"], residual=s["res"], dropout=s["p"], seed=s["seed"],
                       offset=s["offset"], save_preact=s["save"])
        return {"y": y[0], "z": y[1]} if s["save"] else {"y": y}
    if s["op"] == "linear_backward":
        dx, dw, db = oz2.linear_backward(s["dy"], s["x"], s["w"], preact=s["z"], activation=s["act"], dropout=s["p"],
                                         seed=s["seed"], offset=s["offset"])
        return {"dx": dx, "dw": dw, "db": db}
    if s["op"] == "dropout":
        if s["backward"]:
            return oz2.dropout_backward(s["x"], s["p"], seed=s["seed"], offset=s["offset"])
        return oz2.dropout(s["x"], s["p"], seed=s["seed"], offset=s["offset"], residual=s["res"])
    if s["backward"]:
        dq, dk, dwq, dwk = oz2.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"],
                                                     s["pos"], eps=EPS, interleaved=s["interleaved"])
        return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    q, k = oz2.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["pos"], eps=EPS,
                            interleaved=s["interleaved"])
    return {"q": q, "k": k}


def run(state):
    if own:
        return _run_own(state)
    return {"linear": _linear_plain, "linear_backward": _linear_backward_plain, "dropout": _dropout_plain,
            "qk_norm_rope": _qk_plain}[state["op"]](state)


# ------------------------------------------------------------------ 64 bits
def _exact_factor(rows, cols, p, seed, offset):
    """keep / (1 - p) as a float64 matrix; the generator in numpy's unsigned 64-bit words."""
    t = int(math.floor(65536 * p + 0.5))
    if t == 0:
        return 1.0
    low, u = np.uint64(0xFFFFFFFF), np.uint64
    block = np.empty((4, rows, -(-cols // 8)), np.uint64)
    block[0], block[1] = np.arange(block.shape[2], dtype=np.uint64), np.arange(rows, dtype=np.uint64)[:, None]
    block[2], block[3] = u(offset % 2**32), u(offset // 2**32)
    for r in range(7):
        left, right = block[0] * u(0xD2511F53), block[2] * u(0xCD9E8D57)
        key = [u((seed // 2**(32 * i) + r * step) % 2**32) for i, step in enumerate((0x9E3779B9, 0xBB67AE85))]
        block[0], block[2] = (right >> u(32)) ^ block[1] ^ key[0], (left >> u(32)) ^ block[3] ^ key[1]
        block[1], block[3] = right & low, left & low
    draws = np.ascontiguousarray(np.moveaxis(block, 0, -1).astype("<u4")).view("<u2").reshape(rows, -1)[:, :cols]
    return torch.from_numpy(draws >= t).cuda().double() * (1.0 / (1.0 - t / 65536.0))


def _exact_act(z, act):
    """act(z) and act'(z), gelu_tanh by its tanh."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if act == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z * z / 2) * (2 * math.pi) ** -0.5
    t = torch.tanh(GELU_C * (z + GELU_A * z**3))
    return z * (1 + t) / 2, (1 + t) / 2 + z * (1 - t * t) / 2 * GELU_C * (1 + 3 * GELU_A * z * z)


def _exact_norm_rope(x, w, cos, sin, interleaved):
    """The whole map as torch's own float64 operations that autograd follows; the rotation as complex products."""
    u = x * w / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS)
    half = cos.shape[1]
    turn = torch.complex(cos.double(), sin.double())[:, None]
    if interleaved:
        v = torch.view_as_real(torch.view_as_complex(u[..., :2 * half].unflatten(-1, (half, 2)).contiguous()) * turn).flatten(-2)
    else:
        c = torch.complex(u[..., :half], u[..., half:2 * half]) * turn
        v = torch.cat((c.real, c.imag), -1)
    return torch.cat((v, u[..., 2 * half:]), -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("linear", "linear_backward"):
        x, w = s["x"].double(), s["w"].double()
        factor = _exact_factor(case["m"], case["n"], case["p"], s["seed"], s["offset"])
        if case["op"] == "linear_backward":
            dz = s["dy"].double() * factor
            if s["z"] is not None:
                dz = dz * _exact_act(s["z"].double(), case["act"])[1]
            return {"dx": torch.mm(dz, w), "dw": torch.mm(dz.t(), x), "db": dz.sum(0)}
        z = torch.mm(x, w.t())
        if s["b"] is not None:
            z = z + s["b"].double()
        y = _exact_act(z, case["act"])[0] * factor
        if s["res"] is not None:
            y = y + s["res"].double()
        return {"y": y, "z": z} if case["save"] else {"y": y}
    if case["op"] == "dropout":
        y = s["x"].double() * _exact_factor(case["m"], case["n"], case["p"], s["seed"], s["offset"])
        return y if s["res"] is None else y + s["res"].double()
    cos, sin = s["cos"][s["pos"]], s["sin"][s["pos"]]
    leaves = [s[name].double().requires_grad_(case["backward"]) for name in ("q", "k", "wq", "wk")]
    q, k, wq, wk = leaves
    q_out = _exact_norm_rope(q, wq, cos, sin, case["interleaved"])
    k_out = _exact_norm_rope(k, wk, cos, sin, case["interleaved"])
    if not case["backward"]:
        return {"q": q_out, "k": k_out}
    dq, dk, dwq, dwk = torch.autograd.grad((q_out, k_out), leaves, (s["dq"].double(), s["dk"].double()))
    return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
