"""Host-side checks of the layer operators that need no GPU: every declared entry
point is exported, argument errors come back before any device work, a machine
without a GPU gets a loud error, and the generator of the 64-bit definitions
spreads its draws evenly."""
import ctypes
import os
import re

import numpy as np
import pytest

import emulated_fp64_gemm_gb300 as oz2
from emulated_fp64_gemm_gb300 import _build
from tests._util import ROOT

torch = pytest.importorskip("torch")
from emulated_fp64_gemm_gb300 import layers  # noqa: E402
from tests._layers_ref import keep_mask, philox  # noqa: E402

INVALID, CUDA = 1, 4
P = ctypes.c_void_p(16)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return layers._library()


def test_exports_every_declared_symbol(lib):
    text = open(os.path.join(ROOT, "include", "ozaki2_layers.h")).read()
    names = set(re.findall(r"\b(ozaki2_\w+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S)))
    assert len(names) == 5
    for n in names:
        assert hasattr(lib, n), n
    for name in layers.__all__:
        assert getattr(oz2, name) is getattr(layers, name) and name in oz2.__all__
    enum = dict((k.lower(), int(v)) for k, v in re.findall(r"\bOZ2_ACT_(\w+)\s*=\s*(\d+)", text))
    assert enum == oz2.ACTIVATIONS


def linear(lib, m=4, k=8, n=8, x=P, ldx=8, w=P, ldw=8, bias=None, res=None, ldr=8, y=P, ldy=8, z=None, ldz=8, dtype=0, act=0,
           p=0.0):
    return lib.ozaki2_linear(m, k, n, x, ldx, w, ldw, bias, res, ldr, y, ldy, z, ldz, dtype, act, p, 1, 2, None)


def backward(lib, m=4, k=8, n=8, dy=P, lddy=8, x=P, ldx=8, w=P, ldw=8, z=P, ldz=8, dx=P, lddx=8, dw=P, lddw=8, db=P, dtype=0,
             act=2, p=0.0):
    return lib.ozaki2_linear_backward(m, k, n, dy, lddy, x, ldx, w, ldw, z, ldz, dx, lddx, dw, lddw, db, dtype, act, p, 1, 2,
                                      None)


def drop(lib, rows=4, cols=8, x=P, ldx=8, res=None, ldr=8, y=P, ldy=8, dtype=0, p=0.1):
    return lib.ozaki2_dropout(rows, cols, x, ldx, res, ldr, y, ldy, dtype, p, 1, 2, None)


def qk(lib, tokens=4, dim=16, rot=16, q=None, k=None, wq=P, cos=P, pos=P, eps=1e-6, dtype=0, q_out=None, rows=4):
    h = layers._Heads
    q, k, q_out = q or h(16, 2, 32, 16), k or h(16, 1, 16, 16), q_out or h(16, 2, 32, 16)
    return lib.ozaki2_qk_norm_rope(tokens, dim, rot, q, k, wq, P, cos, P, rows, pos, eps, 0, dtype, q_out, h(16, 1, 16, 16), None)


def test_argument_errors_come_before_any_device_work(lib):
    for f, cases in (
        (linear, [dict(m=-1), dict(k=-1), dict(n=2**31), dict(x=None), dict(w=None), dict(y=None), dict(ldx=7), dict(ldw=7),
                  dict(ldy=7), dict(res=P, ldr=7), dict(z=P, ldz=7), dict(dtype=2), dict(dtype=-1), dict(act=5), dict(act=-1),
                  dict(p=-0.1), dict(p=1.1), dict(p=float("nan"))]),
        (backward, [dict(m=-1), dict(dy=None), dict(lddy=7), dict(x=None), dict(w=None), dict(z=None), dict(ldz=7), dict(lddx=7),
                    dict(lddw=7), dict(dtype=2), dict(act=9), dict(p=2.0)]),
        (drop, [dict(rows=-1), dict(cols=2**31), dict(x=None), dict(y=None), dict(ldx=7), dict(ldy=7), dict(res=P, ldr=7),
                dict(dtype=3), dict(p=float("nan"))]),
        (qk, [dict(tokens=-1), dict(dim=0), dict(dim=513), dict(dim=2**33), dict(rot=17), dict(rot=3), dict(rot=-2), dict(wq=None),
              dict(cos=None), dict(pos=None), dict(eps=-1.0), dict(eps=float("nan")), dict(dtype=3), dict(rows=-1),
              dict(q=layers._Heads(None, 2, 32, 16)), dict(q=layers._Heads(16, -1, 32, 16)),
              dict(q=layers._Heads(16, 2, -32, 16)), dict(q_out=layers._Heads(16, 3, 32, 16)),
              dict(q_out=layers._Heads(None, 2, 32, 16))]),
    ):
        for kw in cases:
            assert f(lib, **kw) == INVALID, (f.__name__, kw)


def test_no_gpu_means_a_loud_error(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert linear(lib) == CUDA and backward(lib) == CUDA and drop(lib) == CUDA and qk(lib) == CUDA
    x = torch.zeros(2, 8, dtype=torch.bfloat16)
    for f in (lambda: oz2.linear(x, x), lambda: oz2.linear_backward(x, x, x), lambda: oz2.dropout(x, 0.1, seed=1)):
        with pytest.raises(ValueError):
            f()


def test_row_major_views_pass_through_and_others_are_copied():
    base = torch.arange(60.0).reshape(6, 10)
    for t, ld in ((base, 10), (base[1:4, 2:7], 10), (base[:1, :5], 5), (base[:, :1], 10), (base[:0], 10), (base.t()[:, :1][:1], 1)):
        got, lead = layers._rows(t)
        assert got is t and (lead == ld or t.shape[0] <= 1)
    for t in (base.t(), base[:, ::2], base[:1].expand(4, 10), base.flip(0).t()):
        got, lead = layers._rows(t)
        assert got is not t and torch.equal(got, t) and lead == t.shape[1]


def test_generator_and_mask_definition():
    # every bit of the counter and of the key changes about half of the output's bits
    base = philox((0, 0, 0, 0), (0, 0))
    for word in range(6):
        for bit in (0, 7, 31):
            c = [0] * 6
            c[word] = 1 << bit
            other = philox(c[:4], c[4:])
            flipped = sum(bin(a ^ b).count("1") for a, b in zip(base, other))
            assert 32 <= flipped <= 96
    for p in (0.0, 0.1, 0.5, 1.0):
        keep, scale = keep_mask(64, 1001, p, 3, 4)
        q = round(65536 * p) / 65536
        assert abs(float(keep.double().mean()) - (1 - q)) <= 6 * np.sqrt(q * (1 - q) / keep.numel()) + 1e-12
        assert scale == (1 / (1 - q) if q < 1 else 0.0)
    # the mask of a wider matrix contains the narrower one's
    a, _ = keep_mask(5, 40, 0.5, 3, 4)
    b, _ = keep_mask(3, 17, 0.5, 3, 4)
    assert torch.equal(a[:3, :17], b)
