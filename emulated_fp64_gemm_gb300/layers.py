"""Layer operators of libozaki2: the dense layers of a transformer block.

``linear`` (product, bias, activation, dropout and residual in one pass) and
its gradients, ``dropout`` from a counter-based generator whose mask is never
stored, and ``qk_norm_rope`` (per-head RMS norm with the position rotation)
and its gradients.  As in the rest of the package this module only checks and
marshals arguments; the work is done by the CUDA kernels behind
``include/ozaki2_layers.h``, which states the formulas, and there is no CPU
fallback.

Matrices are row-major: a (rows, cols) tensor with strides (ld, 1), ld >= cols,
is passed as is, any other layout is first copied.  All calls are asynchronous
on `stream` (default: the tensors' device's current stream).  With a `stream`
given, outputs are allocated for it, and the tensors' memory is kept until its
work is done; ordering it after the inputs' producers is the caller's, as
for any torch operation.  Outputs carry no autograd history; a tensor given
as `out` counts as modified, so that autograd refuses to use what was saved of
it before.

A call of a small layer is bound by the host, so the checks are written out
and the arguments go over as one packed structure: 20 of them one by one
through ctypes take 2.1 us on the Grace host, packed 0.3 us.
"""
from __future__ import annotations

import ctypes
import struct

import torch

__all__ = ["ACTIVATIONS", "linear", "linear_backward", "dropout", "dropout_backward", "qk_norm_rope",
           "qk_norm_rope_backward"]

ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
HEAD_DIM_MAX = 512
_FLOATS = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_HALVES = {torch.bfloat16: 0, torch.float16: 1}
_MASK64 = (1 << 64) - 1

# the argument structures of include/ozaki2_layers.h, field by field
_LINEAR_ARGS = struct.Struct("@qqqPqPqPPqPqPqQQdii")
_LINEAR_BACKWARD_ARGS = struct.Struct("@qqqPqPqPqPqPqPqPQQdii")
_DROPOUT_ARGS = struct.Struct("@qqPqPqPqQQdii")
_HEADS = "Pqqq"
_QK_ARGS = struct.Struct("@qqqqPPP" + 4 * _HEADS + "PP" + 2 * _HEADS + "PPdii")
_QK_FORWARD_ARGS = struct.Struct("@qqqqPPP" + 4 * _HEADS + f"PP{struct.calcsize('@' + 2 * _HEADS + 'PP')}xdii")  # no gradients

_lib = None
# the current stream's handle without the Stream object around it (0.1 instead of 3 us)
_stream_of = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
# autograd learns of a write to a caller's tensor by its version
_written = torch.autograd.graph.increment_version


def _library():
    global _lib
    if _lib is None:
        from . import load_library

        lib = load_library()
        for name in ("linear", "linear_backward", "dropout", "qk_norm_rope", "qk_norm_rope_backward"):
            f = getattr(lib, "ozaki2_" + name)
            f.argtypes, f.restype = [ctypes.c_char_p, ctypes.c_void_p], ctypes.c_int
        _lib = lib
    return _lib


def _fail(code, what):
    from . import Ozaki2Error

    raise Ozaki2Error(code, what)


def _elsewhere(op, device, stream, tensors, *args, **kwargs):
    """op(*args) on the tensors' device and on `stream`, its allocations included."""
    if stream is None:
        with torch.cuda.device(device):
            return op(*args, **kwargs)
    if stream.device_index != device:
        raise ValueError(f"stream is on device {stream.device_index}, the tensors on {device}")
    with torch.cuda.stream(stream):
        result = op(*args, **kwargs)
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return result


def _refuse(name, t, dims, dtypes):
    """The error of a first tensor that is not one of `dtypes`, of `dims` dimensions and on a GPU."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {', '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got shape {tuple(t.shape)}")
    raise ValueError(f"{name} must be a CUDA tensor")


def _check(name, t, dtype, device, shape):
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _ld(t):
    """Leading dimension of a 2-D tensor that is row-major, else 0.  The stride of a size-1 dimension is not used."""
    s0, s1 = t.stride()
    rows, cols = t.shape
    if s1 != 1 and cols > 1:
        return 0
    if rows <= 1:
        return cols or 1
    return s0 if s0 >= cols else 0


def _rows(t, cols):
    """(a row-major tensor of the same values, its leading dimension); cols: t's."""
    if t.is_contiguous():
        return t, cols
    ld = _ld(t)
    if ld == 0 and cols > 0:
        return t.contiguous(), cols
    return t, ld


def _check_out(name, t, dtype, device, shape):
    _check(name, t, dtype, device, shape)
    if _ld(t) == 0 and t.shape[1] > 0:
        raise ValueError(f"{name} must be row-major (strides (ld, 1), ld >= columns), got strides {t.stride()}")


def _activation(name) -> int:
    act = ACTIVATIONS.get(name)
    if act is None:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, got {name!r}")
    return act


def _probability(p) -> float:
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"a dropout probability lies in [0, 1], got {p}")
    return p


def linear(x, w, bias=None, *, activation="none", residual=None, dropout=0.0, seed=0, offset=0, save_preact=False, out=None,
           stream=None):
    """residual + keep * act(x @ w.T + bias) / (1 - dropout), and with `save_preact` also z = x @ w.T + bias.

    x (m, k), w (n, k), bias (n,), residual (m, n): bfloat16 or float16, one
    type.  `out` may be `residual`.  The mask is a function of (row, column,
    seed, offset), the same as `dropout`'s; give each layer and step an offset
    of its own."""
    dtype, device = x.dtype, x.get_device()
    if dtype not in _HALVES or x.dim() != 2 or device < 0:
        _refuse("x", x, 2, _HALVES)
    m, k = x.shape
    if w.dim() != 2:
        raise ValueError(f"w must have shape (n, {k}), got {tuple(w.shape)}")
    n = w.shape[0]
    _check("w", w, dtype, device, (n, k))
    if bias is not None:
        _check("bias", bias, dtype, device, (n,))
    if residual is not None:
        _check("residual", residual, dtype, device, (m, n))
    if out is not None:
        _check_out("out", out, dtype, device, (m, n))
    act = _activation(activation)
    if stream is not None or device != _current_device():
        return _elsewhere(linear, device, stream, (x, w, bias, residual, out), x, w, bias, activation=activation,
                          residual=residual, dropout=dropout, seed=seed, offset=offset, save_preact=save_preact, out=out)

    x, ldx = _rows(x, k)
    w, ldw = _rows(w, k)
    b = r = z = ldr = 0
    if bias is not None:
        if n > 1 and bias.stride(0) != 1:
            bias = bias.contiguous()
        b = bias.data_ptr()
    if residual is not None:
        residual, ldr = _rows(residual, n)
        r = residual.data_ptr()
    if out is not None:
        y, ldy = out, _ld(out)
    else:
        # like the residual where there is one: 0.7 us less on the Grace host
        y = torch.empty_like(residual) if r and residual.is_contiguous() else torch.empty((m, n), dtype=dtype, device=x.device)
        ldy = n
    if save_preact:
        preact = torch.empty((m, n), dtype=dtype, device=x.device) if out is not None else torch.empty_like(y)
        z = preact.data_ptr()
    code = _library().ozaki2_linear(
        _LINEAR_ARGS.pack(m, k, n, x.data_ptr(), ldx, w.data_ptr(), ldw, b, r, ldr, y.data_ptr(), ldy, z, n, seed & _MASK64,
                          offset & _MASK64, _probability(dropout), _HALVES[dtype], act), _stream_of(device))
    if code:
        _fail(code, "ozaki2_linear")
    if out is not None:
        _written(out)
    return (y, preact) if save_preact else y


def linear_backward(dy, x, w, *, preact=None, activation="none", dropout=0.0, seed=0, offset=0, need_dx=True, need_dw=True,
                    need_dbias=True, stream=None):
    """(dx, dw, dbias) of `linear` from dy, the gradient of its output (None for each one that is not needed).

    `preact` is the z that `linear(..., save_preact=True)` returned (not used
    without an activation); activation, dropout, seed and offset are those of
    the forward call.  The gradient of its residual is dy itself."""
    dtype, device = dy.dtype, dy.get_device()
    if dtype not in _HALVES or dy.dim() != 2 or device < 0:
        _refuse("dy", dy, 2, _HALVES)
    m, n = dy.shape
    if x.dim() != 2:
        raise ValueError(f"x must have shape ({m}, k), got {tuple(x.shape)}")
    k = x.shape[1]
    _check("x", x, dtype, device, (m, k))
    _check("w", w, dtype, device, (n, k))
    act = _activation(activation)
    if not act:
        preact = None
    elif preact is None:
        raise ValueError(f"activation {activation!r} needs preact, the saved x @ w.T + bias")
    else:
        _check("preact", preact, dtype, device, (m, n))
    if stream is not None or device != _current_device():
        return _elsewhere(linear_backward, device, stream, (dy, x, w, preact), dy, x, w, preact=preact, activation=activation,
                          dropout=dropout, seed=seed, offset=offset, need_dx=need_dx, need_dw=need_dw, need_dbias=need_dbias)

    # outputs like the inputs they belong to where those are contiguous: 0.7 us less each on the Grace host
    dx = dw = db = None
    if need_dx:
        dx = torch.empty_like(x) if x.is_contiguous() else torch.empty((m, k), dtype=dtype, device=x.device)
    if need_dw:
        dw = torch.empty_like(w) if w.is_contiguous() else torch.empty((n, k), dtype=dtype, device=x.device)
    if need_dbias:
        db = torch.empty((n,), dtype=dtype, device=x.device)
    dy, ldy = _rows(dy, n)
    x, ldx = _rows(x, k)
    w, ldw = _rows(w, k)
    z = ldz = 0
    if preact is not None:
        preact, ldz = _rows(preact, n)
        z = preact.data_ptr()
    code = _library().ozaki2_linear_backward(
        _LINEAR_BACKWARD_ARGS.pack(m, k, n, dy.data_ptr(), ldy, x.data_ptr(), ldx, w.data_ptr(), ldw, z, ldz,
                                   dx.data_ptr() if need_dx else 0, k, dw.data_ptr() if need_dw else 0, k,
                                   db.data_ptr() if need_dbias else 0, seed & _MASK64, offset & _MASK64,
                                   _probability(dropout), _HALVES[dtype], act), _stream_of(device))
    if code:
        _fail(code, "ozaki2_linear_backward")
    return dx, dw, db


def dropout(x, p, *, seed, offset=0, residual=None, out=None, stream=None):
    """residual + keep * x / (1 - p) for x (rows, cols), bfloat16, float16 or float32.

    `out` may be x or residual.  An element's draw is a function of (row,
    column, seed, offset), so the mask can be formed again and is never stored."""
    dtype, device = x.dtype, x.get_device()
    if dtype not in _FLOATS or x.dim() != 2 or device < 0:
        _refuse("x", x, 2, _FLOATS)
    shape = x.shape
    if residual is not None:
        _check("residual", residual, dtype, device, shape)
    if out is not None:
        _check_out("out", out, dtype, device, shape)
    if stream is not None or device != _current_device():
        return _elsewhere(dropout, device, stream, (x, residual, out), x, p, seed=seed, offset=offset, residual=residual, out=out)

    rows, cols = shape
    like = x.is_contiguous()
    x, ldx = _rows(x, cols)
    r = ldr = 0
    if residual is not None:
        residual, ldr = _rows(residual, cols)
        r = residual.data_ptr()
    if out is not None:
        y, ldy = out, _ld(out)
    else:
        y, ldy = torch.empty_like(x) if like else torch.empty(shape, dtype=dtype, device=x.device), cols
    code = _library().ozaki2_dropout(
        _DROPOUT_ARGS.pack(rows, cols, x.data_ptr(), ldx, r, ldr, y.data_ptr(), ldy, seed & _MASK64, offset & _MASK64,
                           _probability(p), _FLOATS[dtype], 0), _stream_of(device))
    if code:
        _fail(code, "ozaki2_dropout")
    if out is not None:
        _written(out)
    return y


def dropout_backward(dy, p, *, seed, offset=0, out=None, stream=None):
    """The gradient of `dropout`'s x: the same mask and scale on dy (the residual's gradient is dy itself)."""
    return dropout(dy, p, seed=seed, offset=offset, out=out, stream=stream)


def _heads(t):
    """(t, strides of its tokens and heads); a copy where the features of a head are not neighbours in memory."""
    s0, s1, s2 = t.stride()
    if s2 != 1 and t.shape[2] > 1:
        t = t.contiguous()
        s0, s1, _ = t.stride()
    return t, s0, s1


def _check_heads_out(name, t, like):
    _check(name, t, like.dtype, like.get_device(), like.shape)
    if t.shape[2] > 1 and t.stride(2) != 1 or any(s == 0 and n > 1 for n, s in zip(t.shape, t.stride())):
        raise ValueError(f"{name}'s features must be neighbours and its heads apart, got strides {t.stride()}")


def _check_qk(q, k, q_weight, k_weight, cos, sin, positions, out):
    dtype, device = q.dtype, q.get_device()
    if dtype not in _FLOATS or q.dim() != 3 or device < 0:
        _refuse("q", q, 3, _FLOATS)
    if k.dim() != 3:
        raise ValueError(f"k must have 3 dimensions, got shape {tuple(k.shape)}")
    tokens, nq, dim = q.shape
    nk = k.shape[1]
    if not 1 <= dim <= HEAD_DIM_MAX:
        raise ValueError(f"heads have 1 to {HEAD_DIM_MAX} features, got {dim}")
    _check("k", k, dtype, device, (tokens, nk, dim))
    _check("q_weight", q_weight, dtype, device, (dim,))
    _check("k_weight", k_weight, dtype, device, (dim,))
    table = cos.shape
    if cos.dim() != 2 or 2 * table[1] > dim:
        raise ValueError(f"cos must have shape (positions, rotated features / 2) with at most {dim} rotated, got {tuple(table)}")
    rows, half = table
    _check("cos", cos, torch.float32, device, table)
    _check("sin", sin, torch.float32, device, table)
    _check("positions", positions, torch.int64, device, (tokens,))
    if out is not None:
        _check_heads_out("out[0]", out[0], q)
        _check_heads_out("out[1]", out[1], k)
    return dtype, device, tokens, nq, nk, dim, rows, half


def _contiguous(*tensors):
    return [t if t.is_contiguous() else t.contiguous() for t in tensors]


def qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions, *, eps=1e-6, interleaved=False, out=None, stream=None):
    """Queries and keys, RMS-normed per head and rotated by their token's position, as (q_out, k_out).

    q (tokens, q heads, dim) and k (tokens, k heads, dim), bfloat16, float16 or
    float32, may be views of one projection's output; q_weight, k_weight (dim,)
    of the same type.  cos, sin (rows, rot / 2) float32 tables and positions
    (tokens,) int64: the first rot features of the normed head are rotated, in
    pairs (i, i + rot / 2), or (2 i, 2 i + 1) if `interleaved`.  A position
    outside the tables gives NaN in that token's outputs.  `out`: a pair of
    tensors, q and k themselves for the operation in place."""
    dtype, device, tokens, nq, nk, dim, rows, half = _check_qk(q, k, q_weight, k_weight, cos, sin, positions, out)
    if stream is not None or device != _current_device():
        tensors = (q, k, q_weight, k_weight, cos, sin, positions, *(out or ()))
        return _elsewhere(qk_norm_rope, device, stream, tensors, q, k, q_weight, k_weight, cos, sin, positions, eps=eps,
                          interleaved=interleaved, out=out)

    if out is None:
        where = q.device
        q_out = torch.empty((tokens, nq, dim), dtype=dtype, device=where)
        k_out = torch.empty((tokens, nk, dim), dtype=dtype, device=where)
        qo_token, ko_token, qo_head, ko_head = nq * dim, nk * dim, dim, dim
    else:
        q_out, k_out = out
        qo_token, qo_head, _ = q_out.stride()
        ko_token, ko_head, _ = k_out.stride()
    q, q_token, q_head = _heads(q)
    k, k_token, k_head = _heads(k)
    if not (cos.is_contiguous() and sin.is_contiguous() and positions.is_contiguous() and q_weight.is_contiguous()
            and k_weight.is_contiguous()):
        cos, sin, positions, q_weight, k_weight = _contiguous(cos, sin, positions, q_weight, k_weight)
    code = _library().ozaki2_qk_norm_rope(
        _QK_FORWARD_ARGS.pack(tokens, dim, 2 * half, rows, cos.data_ptr(), sin.data_ptr(), positions.data_ptr(), q.data_ptr(), nq,
                              q_token, q_head, k.data_ptr(), nk, k_token, k_head, q_out.data_ptr(), nq, qo_token, qo_head,
                              k_out.data_ptr(), nk, ko_token, ko_head, q_weight.data_ptr(), k_weight.data_ptr(), eps,
                              _FLOATS[dtype], 1 if interleaved else 0), _stream_of(device))
    if code:
        _fail(code, "ozaki2_qk_norm_rope")
    if out is not None:
        _written(out)
    return q_out, k_out


def qk_norm_rope_backward(dq_out, dk_out, q, k, q_weight, k_weight, cos, sin, positions, *, eps=1e-6, interleaved=False,
                          out=None, stream=None):
    """(dq, dk, dq_weight, dk_weight) of `qk_norm_rope` from the gradients of its outputs.

    The other arguments are the forward call's.  A token whose position is
    outside the tables gets NaN in dq and dk and adds nothing to the weights'
    gradients.  `out`: a pair of tensors for
    dq and dk, such as the slices of the joined projection's gradient."""
    dtype, device, tokens, nq, nk, dim, rows, half = _check_qk(q, k, q_weight, k_weight, cos, sin, positions, out)
    _check("dq_out", dq_out, dtype, device, (tokens, nq, dim))
    _check("dk_out", dk_out, dtype, device, (tokens, nk, dim))
    if stream is not None or device != _current_device():
        tensors = (dq_out, dk_out, q, k, q_weight, k_weight, cos, sin, positions, *(out or ()))
        return _elsewhere(qk_norm_rope_backward, device, stream, tensors, dq_out, dk_out, q, k, q_weight, k_weight, cos, sin,
                          positions, eps=eps, interleaved=interleaved, out=out)

    where = q.device
    if out is None:
        dq = torch.empty((tokens, nq, dim), dtype=dtype, device=where)
        dk = torch.empty((tokens, nk, dim), dtype=dtype, device=where)
        dq_token, dk_token, dq_head, dk_head = nq * dim, nk * dim, dim, dim
    else:
        dq, dk = out
        dq_token, dq_head, _ = dq.stride()
        dk_token, dk_head, _ = dk.stride()
    dwq = torch.empty((dim,), dtype=dtype, device=where)
    dwk = torch.empty((dim,), dtype=dtype, device=where)
    q, q_token, q_head = _heads(q)
    k, k_token, k_head = _heads(k)
    dq_out, gq_token, gq_head = _heads(dq_out)
    dk_out, gk_token, gk_head = _heads(dk_out)
    if not (cos.is_contiguous() and sin.is_contiguous() and positions.is_contiguous() and q_weight.is_contiguous()
            and k_weight.is_contiguous()):
        cos, sin, positions, q_weight, k_weight = _contiguous(cos, sin, positions, q_weight, k_weight)
    code = _library().ozaki2_qk_norm_rope_backward(
        _QK_ARGS.pack(tokens, dim, 2 * half, rows, cos.data_ptr(), sin.data_ptr(), positions.data_ptr(), q.data_ptr(), nq, q_token,
                      q_head, k.data_ptr(), nk, k_token, k_head, dq.data_ptr(), nq, dq_token, dq_head, dk.data_ptr(), nk, dk_token,
                      dk_head, q_weight.data_ptr(), k_weight.data_ptr(), dq_out.data_ptr(), nq, gq_token, gq_head,
                      dk_out.data_ptr(), nk, gk_token, gk_head, dwq.data_ptr(), dwk.data_ptr(), eps, _FLOATS[dtype],
                      1 if interleaved else 0), _stream_of(device))
    if code:
        _fail(code, "ozaki2_qk_norm_rope_backward")
    if out is not None:
        _written(out)
    return dq, dk, dwq, dwk
