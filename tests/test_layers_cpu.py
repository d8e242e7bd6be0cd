"""Host-side checks of the layer operators that need no GPU: every declared entry
point is exported, argument errors come back before any device work, a machine
without a GPU gets a loud error, and the generator of the 64-bit definitions
spreads its draws evenly."""
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
P = 16  # a pointer that is not null


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


def fields(name):
    """Names and struct codes of an argument structure, as the header declares it."""
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "ozaki2_layers.h")).read(), flags=re.S)
    body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", text).group(1)
    out = []
    for line in body.split(";"):
        line = " ".join(line.split())
        if not line:
            continue
        kind, names = re.match(r"((?:const )?\w+\*?) (.*)", line).groups()
        for n in names.split(","):
            n = n.strip()
            if kind == "oz2_heads":
                out += [(n + "." + f, c) for f, c in fields("oz2_heads")]
            else:
                out.append((n, "P" if kind.endswith("*") else {"int64_t": "q", "uint64_t": "Q", "double": "d", "int32_t": "i"}[kind]))
    return out


def call(lib, what, struct_name, packer, defaults, changes):
    names = fields(struct_name)
    assert "@" + "".join(c for _, c in names) == packer.format
    values = {**{n: 0 for n, _ in names}, **defaults, **changes}
    assert set(values) == {n for n, _ in names}
    return getattr(lib, what)(packer.pack(*(values[n] for n, _ in names)), None)


def linear(lib, **kw):
    return call(lib, "ozaki2_linear", "oz2_linear_args", layers._LINEAR_ARGS,
                dict(m=4, k=8, n=8, x=P, ldx=8, w=P, ldw=8, ldr=8, y=P, ldy=8, ldz=8), kw)


def backward(lib, **kw):
    return call(lib, "ozaki2_linear_backward", "oz2_linear_backward_args", layers._LINEAR_BACKWARD_ARGS,
                dict(m=4, k=8, n=8, dy=P, lddy=8, x=P, ldx=8, w=P, ldw=8, preact=P, ldz=8, dx=P, lddx=8, dw=P, lddw=8, dbias=P,
                     act=2), kw)


def drop(lib, **kw):
    return call(lib, "ozaki2_dropout", "oz2_dropout_args", layers._DROPOUT_ARGS,
                dict(rows=4, cols=8, x=P, ldx=8, ldr=8, y=P, ldy=8, dropout=0.1), kw)


def qk(lib, **kw):
    heads = {}
    for n, h in (("q", 2), ("k", 1), ("q_out", 2), ("k_out", 1), ("dq_out", 2), ("dk_out", 1)):
        heads |= {n + ".data": P, n + ".heads": h, n + ".token_stride": 16 * h, n + ".head_stride": 16}
    base = dict(tokens=4, dim=16, rot=16, table_rows=4, cos=P, sin=P, positions=P, q_weight=P, k_weight=P, dq_weight=P, dk_weight=P,
                eps=1e-6, **heads)
    codes = [call(lib, f, "oz2_qk_args", layers._QK_ARGS, base, kw) for f in ("ozaki2_qk_norm_rope", "ozaki2_qk_norm_rope_backward")]
    assert codes[0] == codes[1]
    return codes[0]


def test_argument_errors_come_before_any_device_work(lib):
    nan = float("nan")
    for f, cases in (
        (linear, [dict(m=-1), dict(k=-1), dict(n=2**31), dict(x=0), dict(w=0), dict(y=0), dict(ldx=7), dict(ldw=7), dict(ldy=7),
                  dict(residual=P, ldr=7), dict(preact=P, ldz=7), dict(dtype=2), dict(dtype=-1), dict(act=5), dict(act=-1),
                  dict(dropout=-0.1), dict(dropout=1.1), dict(dropout=nan)]),
        (backward, [dict(m=-1), dict(dy=0), dict(lddy=7), dict(x=0), dict(w=0), dict(preact=0), dict(ldz=7), dict(lddx=7),
                    dict(lddw=7), dict(dtype=2), dict(act=9), dict(dropout=2.0)]),
        (drop, [dict(rows=-1), dict(cols=2**31), dict(x=0), dict(y=0), dict(ldx=7), dict(ldy=7), dict(residual=P, ldr=7),
                dict(dtype=3), dict(dropout=nan), dict(reserved=1)]),
        (qk, [dict(tokens=-1), dict(dim=0), dict(dim=513), dict(dim=2**33), dict(rot=17), dict(rot=3), dict(rot=-2),
              dict(q_weight=0), dict(cos=0), dict(positions=0), dict(eps=-1.0), dict(eps=nan), dict(dtype=3), dict(table_rows=-1),
              {"q.data": 0}, {"q.heads": -1}, {"q.token_stride": -32}, {"q_out.heads": 3}, {"k_out.data": 0}]),
    ):
        for kw in cases:
            assert f(lib, **kw) == INVALID, (f.__name__, kw)
    for name in ("linear", "linear_backward", "dropout", "qk_norm_rope", "qk_norm_rope_backward"):
        assert getattr(lib, "ozaki2_" + name)(None, None) == INVALID


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
        got, lead = layers._rows(t, t.shape[1])
        assert got is t and (lead == ld or t.shape[0] <= 1)
    for t in (base.t(), base[:, ::2], base[:1].expand(4, 10), base.flip(0).t()):
        got, lead = layers._rows(t, t.shape[1])
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
