"""Operators of libozaki2 around the dense layers: norm, log probabilities and the optimiser's step.

``rms_norm`` (with the residual stream's addition, in the input's type or in
8 bits with scales) and its gradients, ``token_logprobs`` (log probabilities of
given tokens, entropy and the most likely alternatives) and its gradient, and
``adamw`` (one step over many tensors at once, states in 32 or 8 bits).  As in
``layers.py`` this module only checks and marshals arguments; the work is done
by the CUDA kernels behind ``include/ozaki2_steps.h``, which states the
formulas, and there is no CPU fallback.  Matrices, streams, `out` tensors and
autograd are treated as there.
"""
from __future__ import annotations

import ctypes
import struct
from array import array
from operator import attrgetter
from typing import NamedTuple, Optional

import torch

from .layers import (_FLOATS, _check, _check_out, _current_device, _elsewhere, _fail, _HALVES, _ld, _MASK64, _refuse, _rows,
                     _stream_of, _written)

__all__ = ["TokenLogprobs", "AdamWState", "rms_norm", "rms_norm_backward", "token_logprobs", "token_logprobs_backward",
           "adamw_state", "adamw"]

TOP_MAX = 32
ADAMW_BLOCK = 256

# the argument structures of include/ozaki2_steps.h, field by field
_RMS_NORM_ARGS = struct.Struct("@qqPqPqPPqPqPqdii")
_RMS_NORM_BACKWARD_ARGS = struct.Struct("@qqPqPqPPqPqPdii")
_TOKEN_LOGPROBS_ARGS = struct.Struct("@qqPqPqPPPPPPPdii")
_TOKEN_LOGPROBS_BACKWARD_ARGS = struct.Struct("@qqPqPqPPPPPPPPqdii")
_ADAMW_ARGS = struct.Struct("@qPPPPPPPPPPPddddddQiiii")

_lib = None


def _library():
    global _lib
    if _lib is None:
        from . import load_library

        lib = load_library()
        for name in ("rms_norm", "rms_norm_backward", "token_logprobs", "token_logprobs_backward", "adamw"):
            f = getattr(lib, "ozaki2_" + name)
            f.argtypes, f.restype = [ctypes.c_char_p, ctypes.c_void_p], ctypes.c_int
        _lib = lib
    return _lib


def _vector(t):
    return t if t.is_contiguous() else t.contiguous()


# ------------------------------------------------------------------ rms_norm
def rms_norm(x, weight, *, residual=None, eps=1e-6, out_dtype=None, block=None, out=None, residual_out=None, stream=None):
    """s / sqrt(mean(s^2) + eps) * weight for s = x + residual, row by row; with a residual also s, as (y, s).

    x, residual (rows, cols) and weight (cols,): bfloat16, float16 or float32,
    one type.  `out` may be x or residual, `residual_out` too (but not both the
    same).  With `out_dtype` torch.float8_e4m3fn y comes as (q, scale) and stands
    for q * scale: scale (rows, 1) float32 is each row's largest magnitude over
    448, or with `block` 128 that of 128 columns, (rows, ceil(cols / 128)); with a
    residual (q, scale, s)."""
    dtype, device = x.dtype, x.get_device()
    if dtype not in _FLOATS or x.dim() != 2 or device < 0:
        _refuse("x", x, 2, _FLOATS)
    shape = x.shape
    rows, cols = shape
    _check("weight", weight, dtype, device, (cols,))
    if residual is not None:
        _check("residual", residual, dtype, device, shape)
    elif residual_out is not None:
        raise ValueError("residual_out is given without a residual")
    quantize = out_dtype is not None and out_dtype is not dtype
    if quantize and out_dtype is not torch.float8_e4m3fn:
        raise TypeError(f"out_dtype must be {dtype} or {torch.float8_e4m3fn}, got {out_dtype}")
    if block is not None and (not quantize or block != 128):
        raise ValueError(f"block is 128 or None, and only for 8-bit outputs, got {block!r}")
    if quantize and block is None and cols == 0 and rows:
        raise ValueError("rows without columns have no scale")
    if out is not None:
        _check_out("out", out, out_dtype if quantize else dtype, device, shape)
    if residual_out is not None:
        _check_out("residual_out", residual_out, dtype, device, shape)
        if out is not None and out.data_ptr() == residual_out.data_ptr() and rows and cols:
            raise ValueError("out and residual_out must be two tensors")
    if stream is not None or device != _current_device():
        return _elsewhere(rms_norm, device, stream, (x, weight, residual, out, residual_out), x, weight, residual=residual, eps=eps,
                          out_dtype=out_dtype, block=block, out=out, residual_out=residual_out)

    like = x.is_contiguous()
    where = x.device
    x, ldx = _rows(x, cols)
    weight = _vector(weight)
    r = h = s = ldr = ldh = 0
    if residual is not None:
        residual, ldr = _rows(residual, cols)
        r = residual.data_ptr()
        if residual_out is not None:
            stream_out, ldh = residual_out, _ld(residual_out)
        else:
            stream_out, ldh = torch.empty_like(x) if like else torch.empty(shape, dtype=dtype, device=where), cols
        h = stream_out.data_ptr()
    if out is not None:
        y, ldy = out, _ld(out)
    elif quantize:
        y, ldy = torch.empty(shape, dtype=out_dtype, device=where), cols
    else:
        y, ldy = torch.empty_like(x) if like else torch.empty(shape, dtype=dtype, device=where), cols
    if quantize:
        scale = torch.empty((rows, 1 if block is None else -(-cols // block)), dtype=torch.float32, device=where)
        s = scale.data_ptr()
    code = _library().ozaki2_rms_norm(
        _RMS_NORM_ARGS.pack(rows, cols, x.data_ptr(), ldx, r, ldr, weight.data_ptr(), y.data_ptr(), ldy, h, ldh, s, block or 0, eps,
                            _FLOATS[dtype], 1 if quantize else 0), _stream_of(device))
    if code:
        _fail(code, "ozaki2_rms_norm")
    if out is not None:
        _written(out)
    if residual_out is not None:
        _written(residual_out)
    if quantize:
        return (y, scale) if residual is None else (y, scale, stream_out)
    return y if residual is None else (y, stream_out)


def rms_norm_backward(dy, x, weight, *, dresidual=None, eps=1e-6, need_dweight=True, out=None, stream=None):
    """(dx, dweight) of `rms_norm` from dy, the gradient of y, and dresidual, that of s where there was a residual.

    x is what was normed: the forward call's x, or its s where there was a
    residual, and dx is then the gradient of x and of the residual alike.  `out`,
    for dx, may be dy, x or dresidual.  dweight is None without `need_dweight`.
    For an 8-bit y, dy is the gradient of the values that q * scale stands for."""
    dtype, device = dy.dtype, dy.get_device()
    if dtype not in _FLOATS or dy.dim() != 2 or device < 0:
        _refuse("dy", dy, 2, _FLOATS)
    shape = dy.shape
    rows, cols = shape
    _check("x", x, dtype, device, shape)
    _check("weight", weight, dtype, device, (cols,))
    if dresidual is not None:
        _check("dresidual", dresidual, dtype, device, shape)
    if out is not None:
        _check_out("out", out, dtype, device, shape)
    if stream is not None or device != _current_device():
        return _elsewhere(rms_norm_backward, device, stream, (dy, x, weight, dresidual, out), dy, x, weight, dresidual=dresidual, eps=eps,
                          need_dweight=need_dweight, out=out)

    like = dy.is_contiguous()
    dy, ldy = _rows(dy, cols)
    x, ldx = _rows(x, cols)
    weight = _vector(weight)
    d = ldd = 0
    if dresidual is not None:
        dresidual, ldd = _rows(dresidual, cols)
        d = dresidual.data_ptr()
    if out is not None:
        dx, lddx = out, _ld(out)
    else:
        dx, lddx = torch.empty_like(dy) if like else torch.empty(shape, dtype=dtype, device=dy.device), cols
    dw = torch.empty_like(weight) if need_dweight else None
    code = _library().ozaki2_rms_norm_backward(
        _RMS_NORM_BACKWARD_ARGS.pack(rows, cols, dy.data_ptr(), ldy, x.data_ptr(), ldx, weight.data_ptr(), d, ldd, dx.data_ptr(), lddx,
                                     dw.data_ptr() if need_dweight else 0, eps, _FLOATS[dtype], 0), _stream_of(device))
    if code:
        _fail(code, "ozaki2_rms_norm_backward")
    if out is not None:
        _written(out)
    return dx, dw


# ------------------------------------------------------------------ token_logprobs
class _TokenLogprobs(NamedTuple):
    logprobs: torch.Tensor                        # (rows,) log p of each row's target
    z_max: Optional[torch.Tensor] = None          # (rows,) the largest logit / temperature
    log_sum: Optional[torch.Tensor] = None        # (rows,) log of the sum of exp(z - z_max)
    entropy: Optional[torch.Tensor] = None        # (rows,) -sum p log p
    top_logprobs: Optional[torch.Tensor] = None   # (rows, top) the largest log p, falling
    top_ids: Optional[torch.Tensor] = None        # (rows, top) int64, their places


class TokenLogprobs(_TokenLogprobs):
    """What `token_logprobs` returns; None for what was not asked for.

    Beside the tuple's six it has `lse` (rows,), z_max + log_sum.  Log p is z - z_max - log_sum, or z - lse with a
    rounding of lse's size: a program that keeps a single number per row may keep lse, and give its gradient
    TokenLogprobs(logprobs=..., lse=...)."""

    lse = None

    def __new__(cls, logprobs, z_max=None, log_sum=None, entropy=None, top_logprobs=None, top_ids=None, lse=None):
        self = tuple.__new__(cls, (logprobs, z_max, log_sum, entropy, top_logprobs, top_ids))
        self.lse = lse
        return self

    def _replace(self, **changes):
        lse = changes.pop("lse", self.lse)
        new = super()._replace(**changes)
        new.lse = lse
        return new


def _check_targets(logits, targets, device):
    if logits.shape[1] == 0 and logits.shape[0]:
        raise ValueError("logits must have a column at least")
    _check("targets", targets, torch.int64, device, (logits.shape[0],))


def _temperature(t) -> float:
    if not 1e-30 <= t <= 1e30:
        raise ValueError(f"temperature must lie between 1e-30 and 1e30, got {t}")
    return t


def token_logprobs(logits, targets, *, temperature=1.0, top=0, entropy=False, ignore_index=-100, stream=None):
    """A TokenLogprobs of logits (rows, vocab), bfloat16, float16 or float32, and targets (rows,) int64; all of it float32.

    With z = logits / temperature: log p of each row's target, 0 where that is
    `ignore_index` and NaN where it is any other number outside the vocabulary;
    with `entropy` the entropy; with `top` (at most 32) the most likely tokens,
    by their logits, the lowest id first among equal ones.  -inf masks a logit, and so does any z below
    the 32-bit range; a row of those alone has log p -inf and entropy 0, a row with NaN
    or +inf has NaN."""
    dtype, device = logits.dtype, logits.get_device()
    if dtype not in _FLOATS or logits.dim() != 2 or device < 0:
        _refuse("logits", logits, 2, _FLOATS)
    rows, vocab = logits.shape
    _check_targets(logits, targets, device)
    if not 0 <= top <= TOP_MAX or top > vocab and rows:
        raise ValueError(f"top must lie in [0, {min(TOP_MAX, vocab)}], got {top}")
    _temperature(temperature)
    if stream is not None or device != _current_device():
        return _elsewhere(token_logprobs, device, stream, (logits, targets), logits, targets, temperature=temperature, top=top,
                          entropy=entropy, ignore_index=ignore_index)

    where = logits.device
    logits, ld = _rows(logits, vocab)
    targets = _vector(targets)
    # an allocation each, like the first: parts of one are slower to make, 7.8 instead of 4.3 us on the Grace host
    logprobs = torch.empty((rows,), dtype=torch.float32, device=where)
    z_max, log_sum, lse = torch.empty_like(logprobs), torch.empty_like(logprobs), torch.empty_like(logprobs)
    h = top_logprobs = top_ids = None
    at_h = at_top = at_ids = 0
    if entropy:
        h = torch.empty_like(logprobs)
        at_h = h.data_ptr()
    if top:
        top_logprobs = torch.empty((rows, top), dtype=torch.float32, device=where)
        top_ids = torch.empty((rows, top), dtype=torch.int64, device=where)
        at_top, at_ids = top_logprobs.data_ptr(), top_ids.data_ptr()
    code = _library().ozaki2_token_logprobs(
        _TOKEN_LOGPROBS_ARGS.pack(rows, vocab, logits.data_ptr(), ld, targets.data_ptr(), ignore_index, logprobs.data_ptr(), z_max.data_ptr(),
                                  log_sum.data_ptr(), lse.data_ptr(), at_h, at_top, at_ids, temperature, top, _FLOATS[dtype]), _stream_of(device))
    if code:
        _fail(code, "ozaki2_token_logprobs")
    return TokenLogprobs(logprobs, z_max, log_sum, h, top_logprobs, top_ids, lse)


def token_logprobs_backward(dlogprobs, logits, targets, saved, *, dentropy=None, temperature=1.0, ignore_index=-100, out=None,
                            stream=None):
    """The gradient of `token_logprobs`' logits, in their type, from those of its logprobs and, if given, its entropy.

    `saved` is the forward call's TokenLogprobs (with its entropy where
    `dentropy` is given; of z_max, log_sum and lse the first two or the last one
    may be None); logits, targets, temperature and ignore_index are the
    forward call's.  dlogprobs, dentropy (rows,) float32.  `out` may be the logits."""
    dtype, device = logits.dtype, logits.get_device()
    if dtype not in _FLOATS or logits.dim() != 2 or device < 0:
        _refuse("logits", logits, 2, _FLOATS)
    rows, vocab = shape = logits.shape
    _check_targets(logits, targets, device)
    vector = (rows,)
    _check("dlogprobs", dlogprobs, torch.float32, device, vector)
    split = saved.z_max is not None and saved.log_sum is not None
    if not split and saved.lse is None:
        raise ValueError("saved needs z_max and log_sum, or lse")
    for name in ("logprobs", "z_max", "log_sum") if split else ("logprobs", "lse"):
        _check("saved." + name, getattr(saved, name), torch.float32, device, vector)
    if dentropy is not None:
        _check("dentropy", dentropy, torch.float32, device, vector)
        if saved.entropy is None:
            raise ValueError("dentropy needs saved.entropy: the forward call's entropy=True")
        _check("saved.entropy", saved.entropy, torch.float32, device, vector)
    _temperature(temperature)
    if out is not None:
        _check_out("out", out, dtype, device, shape)
    if stream is not None or device != _current_device():
        tensors = (dlogprobs, logits, targets, saved.logprobs, saved.z_max, saved.log_sum, saved.lse, saved.entropy, dentropy, out)
        return _elsewhere(token_logprobs_backward, device, stream, tensors, dlogprobs, logits, targets, saved, dentropy=dentropy,
                          temperature=temperature, ignore_index=ignore_index, out=out)

    like = logits.is_contiguous()
    logits, ld = _rows(logits, vocab)
    targets, dlogprobs = _vector(targets), _vector(dlogprobs)
    logprobs = _vector(saved.logprobs)
    at_max = at_sum = at_lse = h = s = 0
    if split:
        z_max, log_sum = _vector(saved.z_max), _vector(saved.log_sum)
        at_max, at_sum = z_max.data_ptr(), log_sum.data_ptr()
    else:
        lse = _vector(saved.lse)
        at_lse = lse.data_ptr()
    if dentropy is not None:
        dentropy, entropy = _vector(dentropy), _vector(saved.entropy)
        h, s = dentropy.data_ptr(), entropy.data_ptr()
    if out is not None:
        d, ldd = out, _ld(out)
    else:
        d, ldd = torch.empty_like(logits) if like else torch.empty(shape, dtype=dtype, device=logits.device), vocab
    code = _library().ozaki2_token_logprobs_backward(
        _TOKEN_LOGPROBS_BACKWARD_ARGS.pack(rows, vocab, logits.data_ptr(), ld, targets.data_ptr(), ignore_index, dlogprobs.data_ptr(), h,
                                           logprobs.data_ptr(), at_max, at_sum, at_lse, s, d.data_ptr(), ldd, temperature,
                                           _FLOATS[dtype], 0), _stream_of(device))
    if code:
        _fail(code, "ozaki2_token_logprobs_backward")
    if out is not None:
        _written(out)
    return d


# ------------------------------------------------------------------ adamw
class _AdamWTensors(NamedTuple):
    step: torch.Tensor                                # int64 (2,): the steps taken, and 0
    exp_avg: torch.Tensor                             # float32, or float8_e4m3fn
    exp_avg_sq: torch.Tensor                          # float32, or uint8: fourth roots, 0 to 255
    exp_avg_scale: Optional[torch.Tensor] = None      # float32, for every 256 elements of 8-bit states
    exp_avg_sq_scale: Optional[torch.Tensor] = None
    master: Optional[torch.Tensor] = None             # float32: the parameters themselves, where theirs are 16-bit copies


class AdamWState(_AdamWTensors):
    """The states of `adamw`, as flat tensors: tensor i of the call begins where those before it end, each rounded up to
    256 elements.  They are plain tensors, to be saved and loaded like any other.

    One of `adamw_state` knows its parameters' sizes besides, copies and pickles of it too, and `adamw` refuses it for
    other sizes or another order of them.  One that is put together from tensors has none (they may be set); there only
    the length of all is checked.  Parameters of equal sizes are told apart by their order alone."""

    sizes = None  # a list of the parameters' sizes, or None

    def _replace(self, **changes):
        new = super()._replace(**changes)
        new.sizes = self.sizes
        return new


_dtype_of, _device_of = attrgetter("dtype"), torch.Tensor.get_device


def _blocks(sizes):
    return sum([(n + ADAMW_BLOCK - 1) // ADAMW_BLOCK for n in sizes])


def adamw_state(params, *, bits=32, master=False):
    """A fresh AdamWState for these parameters, in their order; with `master`, holding 32-bit copies of 16-bit ones."""
    if bits not in (8, 32):
        raise ValueError(f"bits must be 8 or 32, got {bits!r}")
    params = list(params)
    if not params:
        raise ValueError("there are no parameters")
    device = params[0].device
    sizes = [t.numel() for t in params]
    blocks = _blocks(sizes)
    total = blocks * ADAMW_BLOCK

    def zeros(n, dtype=torch.float32):
        return torch.zeros(n, dtype=dtype, device=device)

    state = AdamWState(zeros(2, torch.int64), zeros(total, torch.float32 if bits == 32 else torch.float8_e4m3fn),
                       zeros(total, torch.float32 if bits == 32 else torch.uint8), *(zeros(blocks) for _ in range(2 if bits == 8 else 0)))
    state.sizes = sizes
    if not master:
        return state
    if any(t.dtype not in _HALVES for t in params):
        raise TypeError("master weights are for 16-bit parameters")
    copies, at = zeros(total), 0
    for t, n in zip(params, sizes):
        copies[at:at + n] = t.detach().reshape(-1)
        at += -(-n // ADAMW_BLOCK) * ADAMW_BLOCK
    return state._replace(master=copies)


def _fits(t, dtype, device, shape):
    return t.dtype is dtype and t.get_device() == device and t.shape == shape and t.is_contiguous()


def _check_state(state, sizes, dtype, device):
    """The states' bits."""
    step, m, v, scale_m, scale_v, master = state
    if state.sizes is not None and state.sizes != sizes:
        raise ValueError("the state is that of parameters of other sizes, or in another order")
    blocks = _blocks(sizes)
    eight = m.dtype is torch.float8_e4m3fn
    wanted = {"step": (step, torch.int64, (2,)), "exp_avg": (m, torch.float8_e4m3fn if eight else torch.float32, (blocks * ADAMW_BLOCK,)),
              "exp_avg_sq": (v, torch.uint8 if eight else torch.float32, (blocks * ADAMW_BLOCK,))}
    if eight:
        wanted["exp_avg_scale"], wanted["exp_avg_sq_scale"] = (scale_m, torch.float32, (blocks,)), (scale_v, torch.float32, (blocks,))
    elif scale_m is not None or scale_v is not None:
        raise ValueError("scales belong to 8-bit states")
    if master is not None:
        if dtype not in _HALVES:
            raise TypeError("master weights are for 16-bit parameters")
        wanted["master"] = (master, torch.float32, (blocks * ADAMW_BLOCK,))
    for name, (t, kind, shape) in wanted.items():
        if t is None or not _fits(t, kind, device, shape):
            if t is None:
                raise ValueError(f"8-bit states need state.{name}")
            _check("state." + name, t, kind, device, shape)
            raise ValueError(f"state.{name} must be contiguous")
    return 8 if eight else 32


def _number(name, v, device):
    """(address, value) of a number that may be in device memory."""
    if type(v) is float or not isinstance(v, torch.Tensor):
        return 0, v
    _check(name, v, torch.float32, device, v.shape)
    if v.numel() != 1:
        raise ValueError(f"{name} must have one element, got shape {tuple(v.shape)}")
    return v.data_ptr(), 0.0


# (one call for each property of all tensors: a tenth of the time of a call of _check for each)
def _types(name, tensors):
    try:
        return set(map(_dtype_of, tensors))
    except AttributeError:
        i = next(i for i, t in enumerate(tensors) if not isinstance(t, torch.Tensor))
        raise TypeError(f"{name}[{i}] must be a tensor, got {type(tensors[i]).__name__}") from None


def adamw(params, grads, state, *, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, grad_scale=1.0, seed=0, stream=None):
    """One AdamW step over all of `params` at once, in place; `state` is that of `adamw_state`, and counts the step.

    params: contiguous tensors of one type, bfloat16, float16 or float32, each
    there once; grads: tensors of as many elements, in the same order, of their
    type or float32 (a parameter without a gradient is left out, of `state` too).
    lr and grad_scale (what the gradients are multiplied with) are numbers, or
    float32 tensors of one element on the device, which a captured call reads anew
    at each replay.  8-bit states are rounded by draws that are a function of (element,
    step, seed).  16-bit parameters without master copies are rounded to nearest at every
    step: small rates want `master`."""
    params, grads = list(params), list(grads)
    n = len(params)
    if n == 0 or len(grads) != n:
        raise ValueError(f"there must be a gradient for each parameter, and one parameter at least: got {n} and {len(grads)}")
    types, grad_types = _types("params", params), _types("grads", grads)
    dtype, device, grad_dtype = params[0].dtype, params[0].get_device(), grads[0].dtype
    if dtype not in _FLOATS or device < 0:
        _refuse("params[0]", params[0], params[0].dim(), _FLOATS)
    if grad_dtype is not dtype and grad_dtype is not torch.float32:
        raise TypeError(f"grads must be {dtype} or {torch.float32}, got {grad_dtype}")
    tensor = torch.Tensor
    if types != {dtype} or grad_types != {grad_dtype}:
        raise TypeError("params must be of one type, and grads of one type")
    if set(map(_device_of, params)) != {device} or set(map(_device_of, grads)) != {device}:
        raise ValueError(f"params and grads must be on cuda:{device}")
    sizes = list(map(tensor.numel, params))
    if list(map(tensor.numel, grads)) != sizes:
        raise ValueError("each gradient must have as many elements as its parameter")
    if not all(map(tensor.is_contiguous, params)):
        raise ValueError("params must be contiguous")
    bits = _check_state(state, sizes, dtype, device)
    lr_at, lr_value = _number("lr", lr, device)
    scale_at, scale_value = _number("grad_scale", grad_scale, device)
    if stream is not None or device != _current_device():
        more = (t for t in (lr, grad_scale) if isinstance(t, tensor))
        return _elsewhere(adamw, device, stream, (*params, *grads, *state, *more), params, grads, state, lr=lr, betas=betas, eps=eps,
                          weight_decay=weight_decay, grad_scale=grad_scale, seed=seed)

    if not all(map(tensor.is_contiguous, grads)):
        grads = [t.contiguous() for t in grads]
    # (a list first: an array takes its elements from an iterator one by one, a third slower)
    arrays = array("q", [*map(tensor.data_ptr, params), *map(tensor.data_ptr, grads), *sizes])
    at = arrays.buffer_info()[0]
    scale_m = scale_v = 0
    if bits == 8:
        scale_m, scale_v = state.exp_avg_scale.data_ptr(), state.exp_avg_sq_scale.data_ptr()
    code = _library().ozaki2_adamw(
        _ADAMW_ARGS.pack(n, at, at + 8 * n, at + 16 * n, state.exp_avg.data_ptr(), state.exp_avg_sq.data_ptr(), scale_m, scale_v,
                         state.master.data_ptr() if state.master is not None else 0, state.step.data_ptr(), lr_at, scale_at, lr_value,
                         betas[0], betas[1], eps, weight_decay, scale_value, seed & _MASK64, _FLOATS[dtype], _FLOATS[grad_dtype], bits, 0), _stream_of(device))
    if code:
        _fail(code, "ozaki2_adamw")
    _written(params)
    _written([t for t in state if t is not None])
