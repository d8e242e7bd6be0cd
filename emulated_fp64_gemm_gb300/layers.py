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
for any torch operation.  Outputs carry no autograd history.
"""
from __future__ import annotations

import ctypes

import torch

__all__ = ["ACTIVATIONS", "linear", "linear_backward", "dropout", "dropout_backward", "qk_norm_rope",
           "qk_norm_rope_backward"]

ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_MASK64 = (1 << 64) - 1
_lib = None


class _Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("heads", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


def _declare(lib) -> None:
    """Argument types of the layer entry points."""
    i64, u64, i32, f64, vp = ctypes.c_int64, ctypes.c_uint64, ctypes.c_int, ctypes.c_double, ctypes.c_void_p
    lib.ozaki2_linear.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, vp, i64, vp, i64, vp, i64, i32, i32, f64, u64, u64, vp]
    lib.ozaki2_linear_backward.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i32, i32,
                                           f64, u64, u64, vp]
    lib.ozaki2_dropout.argtypes = [i64, i64, vp, i64, vp, i64, vp, i64, i32, f64, u64, u64, vp]
    lib.ozaki2_qk_norm_rope.argtypes = [i64, i64, i64, _Heads, _Heads, vp, vp, vp, vp, i64, vp, f64, i32, i32, _Heads, _Heads, vp]
    lib.ozaki2_qk_norm_rope_backward.argtypes = [i64, i64, i64, _Heads, _Heads, _Heads, _Heads, vp, vp, vp, vp, i64, vp, f64,
                                                 i32, i32, _Heads, _Heads, vp, vp, vp]
    for f in (lib.ozaki2_linear, lib.ozaki2_linear_backward, lib.ozaki2_dropout, lib.ozaki2_qk_norm_rope,
              lib.ozaki2_qk_norm_rope_backward):
        f.restype = i32


def _library():
    global _lib
    if _lib is None:
        from . import load_library

        lib = load_library()
        _declare(lib)
        _lib = lib
    return _lib


def _call(f, what, *args):
    code = f(*args)
    if code:
        from . import Ozaki2Error

        raise Ozaki2Error(code, what)


def _on_stream(op, stream, tensors, outputs):
    """op(the stream's handle) on the tensors' device, with allocations for that stream.  `op` returns its outputs."""
    device = next(t for t in tensors if t is not None).device
    if stream is None:
        if device.index == torch.cuda.current_device():
            return op(torch.cuda.current_stream().cuda_stream)
        with torch.cuda.device(device):
            return op(torch.cuda.current_stream().cuda_stream)
    with torch.cuda.stream(stream):
        result = op(stream.cuda_stream)
    for t in (*tensors, *outputs):
        if t is not None:
            t.record_stream(stream)
    return result


def _check_like(name, t, dtype, device, shape=None):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _check_first(name, t, dims, dtypes):
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {', '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got shape {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")


_HALVES = (torch.bfloat16, torch.float16)
_FLOATS = (torch.bfloat16, torch.float16, torch.float32)


def _ld(t):
    """Leading dimension of a 2-D tensor that is row-major, else None.  The stride of a size-1 dimension is not used."""
    s0, s1 = t.stride()
    rows, cols = t.shape
    if cols > 1 and s1 != 1:
        return None
    if rows <= 1:
        return max(cols, 1)
    return s0 if s0 >= cols else None


def _rows(t):
    """(a row-major tensor of the same values, its leading dimension)."""
    ld = _ld(t)
    if ld is None:
        t = t.contiguous()
        ld = max(t.shape[1], 1)
    return t, ld


def _out_ld(name, t):
    ld = _ld(t)
    if ld is None:
        raise ValueError(f"{name} must be row-major (strides (ld, 1), ld >= columns), got strides {t.stride()}")
    return ld


def _activation(name) -> int:
    if name not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, got {name!r}")
    return ACTIVATIONS[name]


def _probability(p) -> float:
    p = float(p)
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
    _check_first("x", x, 2, _HALVES)
    dtype, device = x.dtype, x.device
    m, k = x.shape
    if w.dim() != 2 or w.shape[1] != k:
        raise ValueError(f"w must have shape (n, {k}), got {tuple(w.shape)}")
    n = w.shape[0]
    _check_like("w", w, dtype, device)
    if bias is not None:
        _check_like("bias", bias, dtype, device, (n,))
    if residual is not None:
        _check_like("residual", residual, dtype, device, (m, n))
    if out is not None:
        _check_like("out", out, dtype, device, (m, n))
        _out_ld("out", out)
    act, p = _activation(activation), _probability(dropout)

    def op(handle):
        xs, ldx = _rows(x)
        ws, ldw = _rows(w)
        b = bias if bias is None or bias.stride(0) == 1 or n <= 1 else bias.contiguous()
        r, ldr = (None, 0) if residual is None else _rows(residual)
        y = torch.empty((m, n), dtype=dtype, device=device) if out is None else out
        z = torch.empty((m, n), dtype=dtype, device=device) if save_preact else None
        _call(_library().ozaki2_linear, "ozaki2_linear", m, k, n, xs.data_ptr(), ldx, ws.data_ptr(), ldw,
              None if b is None else b.data_ptr(), None if r is None else r.data_ptr(), ldr, y.data_ptr(), _ld(y),
              None if z is None else z.data_ptr(), max(n, 1), _DTYPES[dtype], act, p, seed & _MASK64, offset & _MASK64, handle)
        return (y, z) if save_preact else y

    return _on_stream(op, stream, (x, w, bias, residual), (out,))


def linear_backward(dy, x, w, *, preact=None, activation="none", dropout=0.0, seed=0, offset=0, need_dx=True, need_dw=True,
                    need_dbias=True, stream=None):
    """(dx, dw, dbias) of `linear` from dy, the gradient of its output (None for each one that is not needed).

    `preact` is the z that `linear(..., save_preact=True)` returned (not used
    without an activation); activation, dropout, seed and offset are those of
    the forward call.  The gradient of its residual is dy itself."""
    _check_first("dy", dy, 2, _HALVES)
    dtype, device = dy.dtype, dy.device
    m, n = dy.shape
    if x.dim() != 2 or x.shape[0] != m:
        raise ValueError(f"x must have shape ({m}, k), got {tuple(x.shape)}")
    k = x.shape[1]
    _check_like("x", x, dtype, device)
    _check_like("w", w, dtype, device, (n, k))
    act, p = _activation(activation), _probability(dropout)
    if act and preact is None:
        raise ValueError(f"activation {activation!r} needs preact, the saved x @ w.T + bias")
    if act:
        _check_like("preact", preact, dtype, device, (m, n))
    else:
        preact = None

    def op(handle):
        g, ldg = _rows(dy)
        xs, ldx = _rows(x)
        ws, ldw = _rows(w)
        z, ldz = (None, 0) if preact is None else _rows(preact)
        dx = torch.empty((m, k), dtype=dtype, device=device) if need_dx else None
        dw = torch.empty((n, k), dtype=dtype, device=device) if need_dw else None
        db = torch.empty((n,), dtype=dtype, device=device) if need_dbias else None
        ptr = lambda t: None if t is None else t.data_ptr()
        _call(_library().ozaki2_linear_backward, "ozaki2_linear_backward", m, k, n, g.data_ptr(), ldg, xs.data_ptr(), ldx,
              ws.data_ptr(), ldw, ptr(z), ldz, ptr(dx), max(k, 1), ptr(dw), max(k, 1), ptr(db), _DTYPES[dtype], act, p,
              seed & _MASK64, offset & _MASK64, handle)
        return dx, dw, db

    return _on_stream(op, stream, (dy, x, w, preact), ())


def dropout(x, p, *, seed, offset=0, residual=None, out=None, stream=None):
    """residual + keep * x / (1 - p) for x (rows, cols), bfloat16, float16 or float32.

    `out` may be x or residual.  An element's draw is a function of (row,
    column, seed, offset), so the mask can be formed again and is never stored."""
    _check_first("x", x, 2, _FLOATS)
    dtype, device = x.dtype, x.device
    rows, cols = x.shape
    if residual is not None:
        _check_like("residual", residual, dtype, device, (rows, cols))
    if out is not None:
        _check_like("out", out, dtype, device, (rows, cols))
        _out_ld("out", out)
    p = _probability(p)

    def op(handle):
        xs, ldx = _rows(x)
        r, ldr = (None, 0) if residual is None else _rows(residual)
        y = torch.empty((rows, cols), dtype=dtype, device=device) if out is None else out
        _call(_library().ozaki2_dropout, "ozaki2_dropout", rows, cols, xs.data_ptr(), ldx, None if r is None else r.data_ptr(),
              ldr, y.data_ptr(), _ld(y), _DTYPES[dtype], p, seed & _MASK64, offset & _MASK64, handle)
        return y

    return _on_stream(op, stream, (x, residual), (out,))


def dropout_backward(dy, p, *, seed, offset=0, out=None, stream=None):
    """The gradient of `dropout`'s x: the same mask and scale on dy (the residual's gradient is dy itself)."""
    return dropout(dy, p, seed=seed, offset=offset, out=out, stream=stream)


def _heads(t):
    """A (tokens, heads, dim) tensor whose features are neighbours (and others copied), as (tensor, C view)."""
    if t.shape[2] > 1 and t.stride(2) != 1:
        t = t.contiguous()
    return t, _Heads(t.data_ptr(), t.shape[1], t.stride(0), t.stride(1))


def _heads_out(name, t, like):
    if t is None:
        return torch.empty(like.shape, dtype=like.dtype, device=like.device)
    _check_like(name, t, like.dtype, like.device, like.shape)
    if t.shape[2] > 1 and t.stride(2) != 1 or any(s == 0 and n > 1 for n, s in zip(t.shape, t.stride())):
        raise ValueError(f"{name}'s features must be neighbours and its heads apart, got strides {t.stride()}")
    return t


def _check_qk(q, k, q_weight, k_weight, cos, sin, positions):
    _check_first("q", q, 3, _FLOATS)
    dtype, device = q.dtype, q.device
    tokens, _, dim = q.shape
    _check_first("k", k, 3, _FLOATS)
    _check_like("k", k, dtype, device, (tokens, k.shape[1], dim))
    _check_like("q_weight", q_weight, dtype, device, (dim,))
    _check_like("k_weight", k_weight, dtype, device, (dim,))
    if not 1 <= dim <= 512:
        raise ValueError(f"heads have 1 to 512 features, got {dim}")
    if cos.dim() != 2 or 2 * cos.shape[1] > dim:
        raise ValueError(f"cos must have shape (positions, rotated features / 2) with at most {dim} rotated, got {tuple(cos.shape)}")
    _check_like("cos", cos, torch.float32, device)
    _check_like("sin", sin, torch.float32, device, cos.shape)
    _check_like("positions", positions, torch.int64, device, (tokens,))


def qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions, *, eps=1e-6, interleaved=False, out=None, stream=None):
    """Queries and keys, RMS-normed per head and rotated by their token's position, as (q_out, k_out).

    q (tokens, q heads, dim) and k (tokens, k heads, dim), bfloat16, float16 or
    float32, may be views of one projection's output; q_weight, k_weight (dim,)
    of the same type.  cos, sin (rows, rot / 2) float32 tables and positions
    (tokens,) int64: the first rot features of the normed head are rotated, in
    pairs (i, i + rot / 2), or (2 i, 2 i + 1) if `interleaved`.  A position
    outside the tables gives NaN in that token's outputs.  `out`: a pair of
    tensors, q and k themselves for the operation in place."""
    _check_qk(q, k, q_weight, k_weight, cos, sin, positions)
    q_out, k_out = (None, None) if out is None else out
    if out is not None:
        q_out, k_out = _heads_out("out[0]", q_out, q), _heads_out("out[1]", k_out, k)

    def op(handle):
        yq = _heads_out("", None, q) if q_out is None else q_out
        yk = _heads_out("", None, k) if k_out is None else k_out
        (qs, qv), (ks, kv) = _heads(q), _heads(k)
        wq, wk, c, s, pos = (t.contiguous() for t in (q_weight, k_weight, cos, sin, positions))
        _call(_library().ozaki2_qk_norm_rope, "ozaki2_qk_norm_rope", q.shape[0], q.shape[2], 2 * cos.shape[1], qv, kv,
              wq.data_ptr(), wk.data_ptr(), c.data_ptr(), s.data_ptr(), cos.shape[0], pos.data_ptr(), eps, interleaved,
              _DTYPES[q.dtype], _heads(yq)[1], _heads(yk)[1], handle)
        return yq, yk

    return _on_stream(op, stream, (q, k, q_weight, k_weight, cos, sin, positions), (q_out, k_out))


def qk_norm_rope_backward(dq_out, dk_out, q, k, q_weight, k_weight, cos, sin, positions, *, eps=1e-6, interleaved=False,
                          out=None, stream=None):
    """(dq, dk, dq_weight, dk_weight) of `qk_norm_rope` from the gradients of its outputs.

    The other arguments are the forward call's.  `out`: a pair of tensors for
    dq and dk, such as the slices of the joined projection's gradient."""
    _check_qk(q, k, q_weight, k_weight, cos, sin, positions)
    _check_like("dq_out", dq_out, q.dtype, q.device, q.shape)
    _check_like("dk_out", dk_out, q.dtype, q.device, k.shape)
    dq, dk = (None, None) if out is None else out
    if out is not None:
        dq, dk = _heads_out("out[0]", dq, q), _heads_out("out[1]", dk, k)

    def op(handle):
        gq = _heads_out("", None, q) if dq is None else dq
        gk = _heads_out("", None, k) if dk is None else dk
        dwq, dwk = torch.empty_like(q_weight), torch.empty_like(k_weight)
        (qs, qv), (ks, kv), (dqs, dqv), (dks, dkv) = _heads(q), _heads(k), _heads(dq_out), _heads(dk_out)
        wq, wk, c, s, pos = (t.contiguous() for t in (q_weight, k_weight, cos, sin, positions))
        _call(_library().ozaki2_qk_norm_rope_backward, "ozaki2_qk_norm_rope_backward", q.shape[0], q.shape[2],
              2 * cos.shape[1], dqv, dkv, qv, kv, wq.data_ptr(), wk.data_ptr(), c.data_ptr(), s.data_ptr(), cos.shape[0],
              pos.data_ptr(), eps, interleaved, _DTYPES[q.dtype], _heads(gq)[1], _heads(gk)[1], dwq.data_ptr(),
              dwk.data_ptr(), handle)
        return gq, gk, dwq, dwk

    return _on_stream(op, stream, (dq_out, dk_out, q, k, q_weight, k_weight, cos, sin, positions), (dq, dk))
