"""Measured cases of the operators around the dense layers: rms_norm, token_logprobs (with their gradients) and adamw.

Each case is one pass through one operator of a training or serving step.
With `own` false, `run` computes it in elementary torch operations in 32 bits,
rounded once at the end; with `own` true it calls the package's operator.
`exact` computes it in 64 bits, by other formulas where there are any.

Definitions that both sides share:

* rms_norm: s = x + residual, y = s w / sqrt(mean(s^2) + eps), and s itself as the new residual; in 8 bits
  q = e4m3(y / scale) with scale = max(1e-30, largest |y|) / 448 of each row or each 128 columns;
* rms_norm_backward: with r = 1 / sqrt(mean(x^2) + eps) and g = dy w, dx = dresidual + r (g - x r^2 mean(g x)),
  dweight = the rows' sum of dy x r;
* token_logprobs: z = logits / temperature, lse = log sum exp z, the target's z - lse (0 where the target is -100),
  entropy -sum p log p, and the largest z - lse with their places, the lowest place first among equals;
  a row without a finite logit has lse and log probabilities -inf and entropy 0;
* token_logprobs_backward: dlogits = (g (onehot - p) - h p (log p + entropy)) / temperature;
* adamw: m = b1 m + (1 - b1) g, v = b2 v + (1 - b2) g^2, p = p (1 - lr wd) - lr m' / (sqrt(v') + eps), m' and v'
  divided by 1 - b^t.  Each tensor's states start at a multiple of 256 elements in flat buffers.  In 8 bits every
  256 elements share a scale: m is e4m3(m / scale), scale = max(1e-36, max |m| / 448); v is a whole number k,
  0 to 255, that stands for scale k^4, scale = max(1e-36, max v / 255^4), rounded up where its place between
  k^4 and (k + 1)^4 is above the element's draw, and to 1 where it would be 0 without being it.  Draws are
  Philox4x32 with 7 rounds (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011),
  counter (element // 8 low, high, step low, high), key (seed low, high), eight 16-bit draws per call, low half
  first.  The codes k are whole numbers on which both sides agree: v is formed by single roundings in 32 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32}
EPS = 1e-6
IGNORED = -100
LR, B1, B2, ADAM_EPS, DECAY = 3e-4, 0.9, 0.999, 1e-8, 0.1


# ------------------------------------------------------------------ cases
def _norm(rows, cols, dtype, residual=False, quantize=False, block=0):
    return {"op": "rms_norm", "rows": rows, "cols": cols, "dtype": dtype, "residual": residual, "quantize": quantize, "block": block}


def _norm_backward(rows, cols, dtype, dresidual=False):
    return {"op": "rms_norm_backward", "rows": rows, "cols": cols, "dtype": dtype, "dresidual": dresidual}


def _logprobs(rows, vocab, dtype, top=0, entropy=False, temperature=1.0, masked=False, backward=False):
    return {"op": "token_logprobs", "rows": rows, "vocab": vocab, "dtype": dtype, "top": top, "entropy": entropy,
            "temperature": temperature, "masked": masked, "backward": backward}


def _adamw(tensors, elements, dtype, grad, bits, master=False):
    return {"op": "adamw", "tensors": tensors, "elements": elements, "dtype": dtype, "grad": grad, "bits": bits, "master": master}


def listed():
    return [
        # one new token: launch latency
        dict(_norm(1, 8192, "bfloat16", residual=True), name="rms_norm, one token"),
        # nothing is a multiple of anything: a pruned layer
        dict(_norm(1003, 2051, "float16", residual=True), name="rms_norm, ragged"),
        # a prompt in front of products in 8 bits
        dict(_norm(8192, 8192, "bfloat16", residual=True, quantize=True, block=128), name="rms_norm, prompt, 8 bits"),
        # a training batch, with the gradient that comes along the residual stream
        dict(_norm_backward(16384, 4096, "bfloat16", dresidual=True), name="rms_norm backward"),
        # a serving batch whose requests ask for the most likely alternatives
        dict(_logprobs(24, 131072, "float32", top=20, entropy=True, temperature=0.7), name="logprobs, serving batch"),
        # scores over a vocabulary of odd size, most of it masked by a grammar in some rows
        dict(_logprobs(517, 50021, "float16", top=5, entropy=True, masked=True), name="logprobs, ragged, masked"),
        # the loss of a training batch
        dict(_logprobs(4096, 131072, "bfloat16", entropy=True), name="logprobs, training"),
        # and its gradient, with a bonus for entropy
        dict(_logprobs(4096, 131072, "bfloat16", entropy=True, backward=True), name="logprobs backward"),
        # one small block's tensors: latency
        dict(_adamw(12, 1 << 20, "float32", "float32", 32), name="adamw, small"),
        # many tensors of odd sizes, in 8 bits beside 32-bit master weights
        dict(_adamw(97, 5000011, "float16", "float16", 8, master=True), name="adamw, ragged, 8 bits"),
        # a model in mixed precision: 16-bit weights and gradients, all else in 32
        dict(_adamw(160, 1 << 28, "bfloat16", "bfloat16", 32, master=True), name="adamw, mixed precision"),
        # a fine-tuning run that saves memory
        dict(_adamw(160, 1 << 29, "bfloat16", "bfloat16", 8), name="adamw, 8 bits"),
    ]


def _size(rng, low, high):
    """A size spread over the logarithm of the range: a multiple of 64, of 8, or any."""
    v = int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))
    step = rng.choice((64, 64, 8, 1))
    if v > step:
        v -= v % step
    return max(low, min(high, v))


def draw(rng):
    op = rng.choice(("rms_norm", "rms_norm_backward", "token_logprobs", "token_logprobs", "adamw"))
    half = rng.choice(("bfloat16", "float16"))
    any_type = rng.choice((half, half, "float32"))
    if op in ("rms_norm", "rms_norm_backward"):
        while True:
            rows, cols = _size(rng, 1, 16384), _size(rng, 64, 16384)
            if rows * cols <= 1 << 26:
                break
        if op == "rms_norm_backward":
            return _norm_backward(rows, cols, any_type, rng.random() < 0.5)
        quantize = rng.random() < 0.4
        return _norm(rows, cols, any_type, rng.random() < 0.7, quantize, rng.choice((0, 128)) if quantize else 0)
    if op == "token_logprobs":
        while True:
            rows, vocab = _size(rng, 1, 8192), _size(rng, 256, 262144)
            if rows * vocab <= 1 << 28:
                break
        temperature = rng.choice((1.0, 1.0, 0.7, 1.3))
        if rng.random() < 0.4:
            return _logprobs(rows, vocab, any_type, 0, rng.random() < 0.5, temperature, rng.random() < 0.3, True)
        top = rng.choice((0, 0, 1, 5, 20)) if rows * vocab <= 1 << 26 else 0
        return _logprobs(rows, vocab, any_type, top, rng.random() < 0.5, temperature, rng.random() < 0.3)
    kind = rng.choice((("float32", "float32", False), (half, half, False), (half, half, True), (half, "float32", True)))
    return _adamw(_size(rng, 1, 200), _size(rng, 4096, 1 << 27), kind[0], kind[1], rng.choice((8, 32)), kind[2])


def _bytes(name):
    return torch.empty(0, dtype=DTYPES[name]).element_size()


def _sizes(case):
    """The tensors' sizes: a few matrices hold most elements, the others are vectors; none a round number."""
    rng = random.Random(case["tensors"] * 1000003 + case["elements"])
    share = [math.exp(rng.uniform(-7.0, 0.0)) for _ in range(case["tensors"])]
    return [max(1, int(case["elements"] * v / sum(share))) for v in share]


def work(case):
    if case["op"] == "adamw":
        n, p, g = sum(_sizes(case)), _bytes(case["dtype"]), _bytes(case["grad"])
        states = 16 if case["bits"] == 32 else 4 + 16 / 256
        return {"bytes": n * (states + g + (8 + p if case["master"] else 2 * p)), "flops": 14.0 * n}
    size = _bytes(case["dtype"])
    if case["op"] == "token_logprobs":
        n, rows = case["rows"] * case["vocab"], case["rows"]
        if case["backward"]:
            return {"bytes": 2 * size * n + rows * (16 + 8 * (1 + case["entropy"])), "flops": (4.0 + 2 * case["entropy"]) * n}
        return {"bytes": size * n + rows * (16 + 4 * case["entropy"] + 12 * case["top"]), "flops": (3.0 + 2 * case["entropy"]) * n}
    n, rows = case["rows"] * case["cols"], case["rows"]
    if case["op"] == "rms_norm_backward":
        return {"bytes": size * (n * (3 + case["dresidual"]) + 2 * case["cols"]), "flops": 12.0 * n}
    out = 1 if case["quantize"] else size
    scales = 0 if not case["quantize"] else 4 * rows * (-(-case["cols"] // case["block"]) if case["block"] else 1)
    return {"bytes": n * (size * (1 + 2 * case["residual"]) + out) + size * case["cols"] + scales, "flops": 5.0 * n}


# ------------------------------------------------------------------ inputs
def _prepare_adamw(s, normal, g):
    sizes = _sizes(s)
    starts = [0]
    for n in sizes:
        starts.append(starts[-1] + -(-n // 256) * 256)
    total = starts[-1]
    inside = torch.zeros(total, dtype=torch.bool, device="cuda")
    for o, n in zip(starts, sizes):
        inside[o:o + n] = True
    gap = ~inside
    # weights and gradients are kept in flat buffers, as a program does that sums its gradients over machines
    master = normal(total, scale=0.03).float().masked_fill_(gap, 0.0)
    grad = normal(total, scale=1e-3).masked_fill_(gap, 0.0)
    s["param_flat"], s["grad_flat"] = master.to(DTYPES[s["dtype"]]), grad.to(DTYPES[s["grad"]])
    s["params"] = [s["param_flat"][o:o + n] for o, n in zip(starts, sizes)]
    s["grads"] = [s["grad_flat"][o:o + n] for o, n in zip(starts, sizes)]
    s["master"] = master if s["master"] else None
    m = normal(total, scale=3e-4).float().masked_fill_(gap, 0.0)
    v = normal(total, scale=1e-3).float().square_().add_(1e-8).masked_fill_(gap, 0.0)
    s["scale_m"] = s["scale_v"] = None
    if s["bits"] == 8:
        s["scale_m"] = (m.view(-1, 256).abs().amax(1) / 448.0).clamp_(min=1e-36)
        s["scale_v"] = (v.view(-1, 256).amax(1) / 255.0**4).clamp_(min=1e-36)
        m = (m.view(-1, 256) / s["scale_m"][:, None]).view(-1).to(torch.float8_e4m3fn)
        v = (v.view(-1, 256) / s["scale_v"][:, None]).view(-1).sqrt_().sqrt_().round_().clamp_(0, 255).to(torch.uint8)
    s["m"], s["v"] = m, v
    s["step"] = torch.tensor([100 + s["seed"] % 50, 0], device="cuda")  # steps taken; the second word is the operator's own
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(scale).to(dtype)

    s = dict(case, seed=(seed * 0x9E3779B97F4A7C15 + 1) % 2**63)
    if case["op"] == "adamw":
        return _prepare_adamw(s, normal, g)
    dtype = DTYPES[case["dtype"]]
    if case["op"] in ("rms_norm", "rms_norm_backward"):
        rows, cols = case["rows"], case["cols"]
        spread = 1.0 + 9.0 * (torch.rand(cols, generator=g, device="cuda") < 0.01)  # a few features are large in every row
        s["x"] = (normal(rows, cols) * spread).to(dtype)
        s["w"] = (1.0 + 0.1 * normal(cols)).to(dtype)
        if case["op"] == "rms_norm_backward":
            s["dy"] = normal(rows, cols, scale=0.01, dtype=dtype)
            s["dres"] = normal(rows, cols, scale=0.01, dtype=dtype) if case["dresidual"] else None
        else:
            s["res"] = (normal(rows, cols) * spread).to(dtype) if case["residual"] else None
        return s
    rows, vocab = case["rows"], case["vocab"]
    logits = normal(rows, vocab, scale=2.5, dtype=dtype)
    likely = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    logits.scatter_(1, likely[:, None], (8.0 + 6.0 * torch.rand(rows, 1, generator=g, device="cuda")).to(dtype))
    other = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    chance = torch.rand(rows, generator=g, device="cuda")
    targets = torch.where(chance < 0.7, likely, other)
    s["targets"] = torch.where(chance > 0.95, IGNORED, targets)
    if case["masked"]:  # a third of the rows keep one token in a hundred, a few of them none
        part = torch.rand(rows, 1, generator=g, device="cuda")
        keep = torch.where(part < 0.03, 0.0, torch.where(part < 0.33, 0.01, 1.0))
        logits.masked_fill_(torch.rand(rows, vocab, generator=g, device="cuda") >= keep, -math.inf)
    s["logits"] = logits
    if case["backward"]:
        s["dlogprob"] = normal(rows, scale=1.0 / rows)
        s["dentropy"] = normal(rows, scale=0.01 / rows) if case["entropy"] else None
        with torch.no_grad():
            s.update(_logprobs_plain(dict(s, top=0)))
    return s


# ------------------------------------------------------------------ plain forms
def _norm_plain(s):
    u = s["x"].float()
    if s["res"] is not None:
        u = u + s["res"].float()
    y = u * torch.rsqrt((u * u).mean(-1, keepdim=True) + EPS) * s["w"].float()
    out = {} if s["res"] is None else {"residual": u.to(s["x"].dtype)}
    if not s["quantize"]:
        return dict(out, y=y.to(s["x"].dtype))
    rows, cols = y.shape
    block = s["block"] or cols
    y = torch.nn.functional.pad(y, (0, -cols % block)).view(rows, -1, block)
    scale = y.abs().amax(-1).clamp(min=1e-30) / 448.0
    q = (y / scale[..., None]).to(torch.float8_e4m3fn).view(rows, -1)[:, :cols]
    return dict(out, q=q, scale=scale)


def _norm_backward_plain(s):
    x, dy = s["x"].float(), s["dy"].float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    g = dy * s["w"].float()
    dx = r * (g - x * (r * r * (g * x).mean(-1, keepdim=True)))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * x * r).sum(0).to(s["x"].dtype)}


def _logprobs_plain(s):
    z = s["logits"].float() / s["temperature"]
    top = z.amax(-1, keepdim=True)
    z = z - torch.where(top > -math.inf, top, 0.0)
    e = torch.exp(z)
    log_sum = torch.log(e.sum(-1, keepdim=True))
    logp = z - torch.where(log_sum > -math.inf, log_sum, 0.0)
    known = s["targets"] != IGNORED
    target = logp.gather(1, torch.where(known, s["targets"], 0)[:, None])[:, 0]
    out = {"logprob": torch.where(known, target, 0.0), "lse": (top + log_sum)[:, 0]}
    if s["entropy"]:
        out["entropy_value"] = -torch.where(e > 0, torch.exp(logp) * logp, 0.0).sum(-1)
    if s["top"]:
        order = torch.sort(logp, dim=-1, descending=True, stable=True)
        out["top_logprobs"], out["top_ids"] = order.values[:, :s["top"]].contiguous(), order.indices[:, :s["top"]].contiguous()
    return out


def _logprobs_backward_plain(s):
    some = s["lse"] > -math.inf
    logp = s["logits"].float() / s["temperature"] - torch.where(some, s["lse"], 0.0)[:, None]
    p = torch.exp(logp)
    known = s["targets"] != IGNORED
    g = torch.where(known & some, s["dlogprob"], 0.0)
    d = -g[:, None] * p
    at = torch.where(known, s["targets"], 0)[:, None]
    d.scatter_(1, at, torch.where(known[:, None], -g[:, None] * torch.expm1(s["logprob"][:, None]), d.gather(1, at)))
    if s["entropy"]:
        d = d - torch.where(p > 0, s["dentropy"][:, None] * p * (logp + s["entropy_value"][:, None]), 0.0)
    return (d / s["temperature"]).to(s["logits"].dtype)


def _draws(elements, step, seed):
    """Eight 16-bit draws for each eight elements, in whole-number torch operations."""
    mask32 = 0xFFFFFFFF
    groups = torch.arange(elements // 8, device="cuda")
    c0, c1 = groups & mask32, groups >> 32
    c2, c3 = (step & mask32).expand_as(groups), (step >> 32).expand_as(groups)
    k0, k1 = seed & mask32, seed >> 32 & mask32
    for _ in range(7):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (b >> 32 & mask32) ^ c1 ^ k0, b & mask32, (a >> 32 & mask32) ^ c3 ^ k1, a & mask32
        k0, k1 = (k0 + 0x9E3779B9) & mask32, (k1 + 0xBB67AE85) & mask32
    return (torch.stack((c0, c0 >> 16, c1, c1 >> 16, c2, c2 >> 16, c3, c3 >> 16), -1) & 0xFFFF).view(-1)


def _codes(v, scale, step, seed):
    """v in whole numbers k of fourth powers; (k * k) * (k * k) and every other step is one rounding in 32 bits."""
    t = (v.view(-1, 256) * (1.0 / scale)[:, None]).view(-1)
    k = torch.sqrt(torch.sqrt(t)).floor_().clamp_(max=255.0)
    k = k - ((k * k) * (k * k) > t).float()
    up = k + 1.0
    k = torch.where((up * up) * (up * up) <= t, up, k).clamp_(max=255.0)
    up, low = k + 1.0, (k * k) * (k * k)
    step_up = (t - low) * 65536.0 > _draws(v.numel(), step, seed).float() * ((up * up) * (up * up) - low)
    k = (k + (step_up | (k == 0) & (t > 0)).float()).clamp_(max=255.0)
    return k.to(torch.uint8)


def _adamw_plain(s):
    t = s["step"][:1] + 1
    c1, c2 = (1.0 - B1 ** t.double()).float(), (1.0 - B2 ** t.double()).float()
    g = s["grad_flat"].float()
    m, v = s["m"].float(), s["v"].float()
    if s["bits"] == 8:
        m = (m.view(-1, 256) * s["scale_m"][:, None]).view(-1)
        v = (((v * v) * (v * v)).view(-1, 256) * s["scale_v"][:, None]).view(-1)
    m = B1 * m + (1 - B1) * g
    v = B2 * v + (1 - B2) * (g * g)
    p = (s["param_flat"] if s["master"] is None else s["master"]).float()
    p = p * (1 - LR * DECAY) - LR * ((m / c1) / (torch.sqrt(v / c2) + ADAM_EPS))
    if s["bits"] == 8:
        s["scale_m"].copy_((m.view(-1, 256).abs().amax(1) * (1.0 / 448.0)).clamp_(min=1e-36))
        s["scale_v"].copy_((v.view(-1, 256).amax(1) * 255.0**-4).clamp_(min=1e-36))
        s["m"].copy_((m.view(-1, 256) * (1.0 / s["scale_m"])[:, None]).view(-1).to(torch.float8_e4m3fn))
        s["v"].copy_(_codes(v, s["scale_v"], t, s["seed"]))
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    if s["master"] is not None:
        s["master"].copy_(p)
    s["param_flat"].copy_(p)
    s["step"][:1] = t
    return _adamw_outputs(s)


def _adamw_outputs(s):
    return {"param": s["param_flat"], "master": s["master"], "m": s["m"], "v": s["v"], "scale_m": s["scale_m"],
            "scale_v": s["scale_v"], "step": s["step"]}


# ------------------------------------------------------------------ the package's operators
def _run_own(s):
    import emulated_fp64_gemm_gb300 as oz2

    if s["op"] == "rms_norm":
        if s["quantize"]:
            out = oz2.rms_norm(s["x"], s["w"], residual=s["res"], eps=EPS, out_dtype=torch.float8_e4m3fn, block=s["block"] or None)
            return dict(zip(("q", "scale", "residual"), out))
        out = oz2.rms_norm(s["x"], s["w"], residual=s["res"], eps=EPS)
        return {"y": out} if s["res"] is None else {"y": out[0], "residual": out[1]}
    if s["op"] == "rms_norm_backward":
        dx, dw = oz2.rms_norm_backward(s["dy"], s["x"], s["w"], dresidual=s["dres"], eps=EPS)
        return {"dx": dx, "dweight": dw}
    if s["op"] == "adamw":
        state = oz2.AdamWState(step=s["step"], exp_avg=s["m"], exp_avg_sq=s["v"], exp_avg_scale=s["scale_m"],
                               exp_avg_sq_scale=s["scale_v"], master=s["master"])
        oz2.adamw(s["params"], s["grads"], state, lr=LR, betas=(B1, B2), eps=ADAM_EPS, weight_decay=DECAY, seed=s["seed"])
        return _adamw_outputs(s)
    if s["backward"]:
        saved = oz2.TokenLogprobs(logprobs=s["logprob"], lse=s["lse"], entropy=s.get("entropy_value"), top_logprobs=None, top_ids=None)
        return oz2.token_logprobs_backward(s["dlogprob"], s["logits"], s["targets"], saved, dentropy=s["dentropy"],
                                           temperature=s["temperature"], ignore_index=IGNORED)
    r = oz2.token_logprobs(s["logits"], s["targets"], temperature=s["temperature"], top=s["top"], entropy=s["entropy"],
                           ignore_index=IGNORED)
    out = {"logprob": r.logprobs, "lse": r.lse}
    if s["entropy"]:
        out["entropy_value"] = r.entropy
    if s["top"]:
        out["top_logprobs"], out["top_ids"] = r.top_logprobs, r.top_ids
    return out


def run(state):
    if own:
        return _run_own(state)
    if state["op"] == "token_logprobs":
        return _logprobs_backward_plain(state) if state["backward"] else _logprobs_plain(state)
    return {"rms_norm": _norm_plain, "rms_norm_backward": _norm_backward_plain, "adamw": _adamw_plain}[state["op"]](state)


# ------------------------------------------------------------------ 64 bits
def _exact_norm(s):
    u = s["x"].double()
    if s["res"] is not None:
        u += s["res"].double()
    y = u / torch.sqrt(torch.linalg.vector_norm(u, dim=-1, keepdim=True) ** 2 / u.shape[1] + EPS) * s["w"].double()
    out = {} if s["res"] is None else {"residual": u}
    if not s["quantize"]:
        return dict(out, y=y)
    block = s["block"] or y.shape[1]
    parts = [part.abs().amax(1, keepdim=True) for part in y.split(block, dim=1)]
    scale = torch.cat(parts, 1).clamp(min=1e-30) / 448
    return dict(out, q=y / scale.repeat_interleave(block, 1)[:, :y.shape[1]], scale=scale)


def _exact_norm_backward(s):
    """By autograd through the definition, in float64."""
    x, w = s["x"].double().requires_grad_(True), s["w"].double().requires_grad_(True)
    y = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[1] + EPS) * w
    dx, dw = torch.autograd.grad(y, (x, w), s["dy"].double())
    return {"dx": dx if s["dres"] is None else dx + s["dres"].double(), "dweight": dw}


def _exact_rows(s, rows):
    """Log probabilities of some rows, each quantity by its own sum."""
    z = s["logits"][rows].double() / s["temperature"]
    lse = torch.logsumexp(z, -1)
    logp = z - torch.where(torch.isfinite(lse), lse, 0.0)[:, None]
    return lse, logp


def _exact_logprobs(s):
    parts = []
    for rows in torch.arange(s["rows"], device="cuda").split(max(1, (1 << 27) // s["vocab"])):
        lse, logp = _exact_rows(s, rows)
        target = s["targets"][rows]
        part = {"lse": lse, "logprob": torch.where(target == IGNORED, 0.0, logp.gather(1, target.clamp(min=0)[:, None])[:, 0])}
        if s["entropy"]:
            part["entropy_value"] = -torch.special.xlogy(logp.exp(), logp.exp()).sum(-1)
        if s["top"]:
            part["top_logprobs"] = torch.topk(logp, s["top"], dim=-1).values
            part["top_ids"] = None
        parts.append(part)
    return {k: None if parts[0][k] is None else torch.cat([part[k] for part in parts]) for k in parts[0]}


def _exact_logprobs_backward(s):
    """The chain rule through the definition, row by row: d/dz of g log p_t + h entropy."""
    out = torch.empty(s["rows"], s["vocab"], dtype=torch.float64, device="cuda")
    for rows in torch.arange(s["rows"], device="cuda").split(max(1, (1 << 27) // s["vocab"])):
        lse, logp = _exact_rows(s, rows)
        p, target = logp.exp(), s["targets"][rows]
        g = torch.where((target == IGNORED) | torch.isinf(lse), 0.0, s["dlogprob"][rows].double())
        d = torch.zeros_like(p).scatter_(1, target.clamp(min=0)[:, None], g[:, None]) - g[:, None] * p
        if s["entropy"]:
            plogp = torch.special.xlogy(p, p)
            d -= s["dentropy"][rows].double()[:, None] * (plogp - p * plogp.sum(-1, keepdim=True))
        out[rows] = d / s["temperature"]
    return out


def _exact_adamw(s):
    t = int(s["step"][0]) + 1
    g = s["grad_flat"].double()
    m, v = s["m"].double(), s["v"].double()
    if s["bits"] == 8:
        m, v = m * s["scale_m"].double().repeat_interleave(256), v.pow(4) * s["scale_v"].double().repeat_interleave(256)
    m, v = m + (1 - B1) * (g - m), v + (1 - B2) * (g.square() - v)
    p = (s["param_flat"] if s["master"] is None else s["master"]).double()
    p = p - LR * DECAY * p - LR / (1 - B1**t) * m / (torch.sqrt(v) / math.sqrt(1 - B2**t) + ADAM_EPS)
    out = {"param": p, "master": None if s["master"] is None else p, "m": m, "v": v, "step": None}
    if s["bits"] == 8:
        out["scale_m"] = (m.view(-1, 256).abs().amax(1) / 448).clamp(min=1e-36)
        out["scale_v"] = (v.view(-1, 256).amax(1) / 255**4).clamp(min=1e-36)
        out["m"], out["v"] = m / out["scale_m"].repeat_interleave(256), None
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "token_logprobs":
        return _exact_logprobs_backward(s) if case["backward"] else _exact_logprobs(s)
    return {"rms_norm": _exact_norm, "rms_norm_backward": _exact_norm_backward, "adamw": _exact_adamw}[case["op"]](s)
