"""Host-side checks of the step operators that need no GPU: every declared entry point is exported,
argument errors come back before any device work, a machine without a GPU gets a loud error, and the
8-bit states' definition rounds as it says."""
import os
import re

import numpy as np
import pytest

import emulated_fp64_gemm_gb300 as oz2
from emulated_fp64_gemm_gb300 import _build
from tests._util import ROOT

torch = pytest.importorskip("torch")
from emulated_fp64_gemm_gb300 import steps  # noqa: E402
from tests import _steps_ref as ref  # noqa: E402

INVALID, CUDA = 1, 4
P = 16  # a pointer that is not null
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return steps._library()


def header():
    return re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "ozaki2_steps.h")).read(), flags=re.S)


def test_exports_every_declared_symbol(lib):
    names = set(re.findall(r"\b(ozaki2_\w+)\s*\(", header()))
    assert names == {"ozaki2_" + n for n in ("rms_norm", "rms_norm_backward", "token_logprobs", "token_logprobs_backward", "adamw")}
    for n in names:
        assert hasattr(lib, n), n
    for name in steps.__all__:
        assert getattr(oz2, name) is getattr(steps, name) and name in oz2.__all__
    constants = dict(re.findall(r"#define OZ2_(TOP_MAX|ADAMW_BLOCK) (\d+)", header()))
    assert constants == {"TOP_MAX": str(steps.TOP_MAX), "ADAMW_BLOCK": str(steps.ADAMW_BLOCK)}


def fields(name):
    """Names and struct codes of an argument structure, as the header declares it."""
    body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", header()).group(1)
    out = []
    for line in body.split(";"):
        line = " ".join(line.split())
        if not line:
            continue
        kind, names = re.match(r"((?:const )?\w+(?:\* const)?) ?(.*)", line).groups()
        for n in names.split(","):
            n = n.strip()
            code = "P" if n.startswith("*") or "*" in kind else {"int64_t": "q", "uint64_t": "Q", "double": "d", "int32_t": "i"}.get(kind, "P")
            out.append((n.lstrip("* "), code))
    return out


def call(lib, what, packer, defaults, changes):
    names = [(n, c) for n, c in fields("oz2_" + what + "_args")]
    assert "@" + "".join(c for _, c in names) == packer.format, names
    values = {**{n: 0 for n, _ in names}, **defaults, **changes}
    assert set(values) == {n for n, _ in names}
    return getattr(lib, "ozaki2_" + what)(packer.pack(*(values[n] for n, _ in names)), None)


def norm(lib, **kw):
    return call(lib, "rms_norm", steps._RMS_NORM_ARGS,
                dict(rows=4, cols=8, x=P, ldx=8, ldr=8, weight=P, y=P, ldy=8, ldo=8, eps=1e-6), kw)


def norm_backward(lib, **kw):
    return call(lib, "rms_norm_backward", steps._RMS_NORM_BACKWARD_ARGS,
                dict(rows=4, cols=8, dy=P, lddy=8, x=P, ldx=8, weight=P, ldd=8, dx=P, lddx=8, dweight=P, eps=1e-6), kw)


def logprobs(lib, **kw):
    return call(lib, "token_logprobs", steps._TOKEN_LOGPROBS_ARGS,
                dict(rows=4, vocab=50, logits=P, ld=50, targets=P, ignore_index=-100, logprobs=P, z_max=P, log_sum=P, temperature=1.0), kw)


def logprobs_backward(lib, **kw):
    return call(lib, "token_logprobs_backward", steps._TOKEN_LOGPROBS_BACKWARD_ARGS,
                dict(rows=4, vocab=50, logits=P, ld=50, targets=P, dlogprobs=P, logprobs=P, z_max=P, log_sum=P, dlogits=P, ldd=50,
                     temperature=1.0), kw)


def tensors(*entries):
    """Columns of (param, grad, elements), each contiguous."""
    return np.ascontiguousarray(np.array(entries, dtype=np.int64).T)


def adamw(lib, table=None, **kw):
    t = tensors((1 << 20, 1 << 30, 1000), (1 << 21, 1 << 31, 7)) if table is None else table
    return call(lib, "adamw", steps._ADAMW_ARGS,
                dict(count=t.shape[1], params=t[0].ctypes.data, grads=t[1].ctypes.data, elements=t[2].ctypes.data, exp_avg=P, exp_avg_sq=P,
                     step=P, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, grad_scale=1.0, dtype=0, grad_dtype=0, bits=32),
                kw)


def test_argument_errors_come_before_any_device_work(lib):
    for f, cases in (
        (norm, [dict(rows=-1), dict(cols=2**31), dict(x=0), dict(y=0), dict(weight=0), dict(ldx=7), dict(ldy=7), dict(residual=P, ldr=7),
                dict(residual_out=P, ldo=7), dict(eps=-1e-9), dict(eps=NAN), dict(eps=INF), dict(dtype=3), dict(dtype=-1),
                dict(quantize=2), dict(quantize=1), dict(quantize=1, scale=P, block=64), dict(block=128), dict(quantize=1, block=128)]),
        (norm_backward, [dict(rows=-1), dict(cols=-1), dict(dy=0), dict(x=0), dict(dx=0), dict(weight=0), dict(lddy=7), dict(ldx=7),
                         dict(lddx=7), dict(dresidual=P, ldd=7), dict(eps=NAN), dict(dtype=3), dict(reserved=1)]),
        (logprobs, [dict(rows=-1), dict(vocab=0), dict(vocab=2**31), dict(logits=0), dict(targets=0), dict(logprobs=0), dict(z_max=0),
                    dict(log_sum=0), dict(ld=49), dict(top=33, top_logprobs=P, top_ids=P), dict(top=-1), dict(top=3),
                    dict(top=3, top_ids=P), dict(vocab=4, top=5, top_logprobs=P, top_ids=P), dict(temperature=0.0),
                    dict(temperature=-1.0), dict(temperature=NAN), dict(temperature=INF), dict(dtype=3)]),
        (logprobs_backward, [dict(rows=-1), dict(vocab=0), dict(logits=0), dict(targets=0), dict(dlogprobs=0), dict(logprobs=0),
                             dict(z_max=0), dict(log_sum=0), dict(dlogits=0), dict(ld=49), dict(ldd=49), dict(dentropy=P),
                             dict(temperature=0.0), dict(dtype=7), dict(reserved=2)]),
        (adamw, [dict(count=-1), dict(params=0), dict(grads=0), dict(elements=0), dict(exp_avg=0), dict(exp_avg_sq=0), dict(step=0), dict(beta1=1.0), dict(beta2=-0.1),
                 dict(beta1=NAN), dict(eps=-1.0), dict(lr=INF), dict(lr=NAN), dict(weight_decay=NAN), dict(grad_scale=INF),
                 dict(dtype=3), dict(grad_dtype=1), dict(bits=16), dict(bits=8), dict(bits=8, exp_avg_scale=P),
                 dict(bits=8, exp_avg_scale=P, exp_avg_sq_scale=P, exp_avg=12), dict(dtype=2, grad_dtype=2, master=P), dict(reserved=1),
                 dict(table=tensors((P, P, -1))), dict(table=tensors((0, P, 1))), dict(table=tensors((P, 0, 1))),
                 dict(table=tensors((P, P, 2**41))),
                 # the same parameter twice, and one inside another
                 dict(table=tensors((1 << 20, P, 100), (1 << 20, P, 100))),
                 dict(table=tensors((1 << 20, P, 100), (1 << 10, P, 10), ((1 << 20) + 198, P, 100)))]),
    ):
        for kw in cases:
            assert f(lib, **kw) == INVALID, (f.__name__, kw)
    for name in ("rms_norm", "rms_norm_backward", "token_logprobs", "token_logprobs_backward", "adamw"):
        assert getattr(lib, "ozaki2_" + name)(None, None) == INVALID


def test_no_gpu_means_a_loud_error(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert norm(lib) == CUDA and norm(lib, quantize=1, scale=P) == CUDA and norm_backward(lib) == CUDA
    assert logprobs(lib) == CUDA and logprobs_backward(lib) == CUDA and adamw(lib) == CUDA
    assert adamw(lib, table=tensors((1 << 20, P, 100), ((1 << 20) + 200, P, 100))) == CUDA  # neighbours do not overlap
    x, w, t = torch.zeros(2, 8), torch.zeros(8), torch.zeros(2, dtype=torch.int64)
    for f in (lambda: oz2.rms_norm(x, w), lambda: oz2.rms_norm_backward(x, x, w), lambda: oz2.token_logprobs(x, t),
              lambda: oz2.token_logprobs_backward(w, x, t, None), lambda: oz2.adamw([x], [x], oz2.adamw_state([x]), lr=1e-3)):
        with pytest.raises(ValueError):
            f()


def test_empty_calls_need_no_device(lib):
    assert norm(lib, rows=0, x=0, y=0) == 0 and norm(lib, cols=0, x=0, y=0, weight=0) == 0
    assert norm_backward(lib, cols=0, dy=0, x=0, dx=0, weight=0) == 0
    assert logprobs(lib, rows=0, logits=0, targets=0, logprobs=0, z_max=0, log_sum=0) == 0
    assert logprobs_backward(lib, rows=0, logits=0, targets=0, dlogprobs=0, logprobs=0, z_max=0, log_sum=0, dlogits=0) == 0


def test_state_layout():
    params = [torch.ones(3, 5, dtype=torch.bfloat16), torch.full((256,), 2.0, dtype=torch.bfloat16), torch.full((257,), 3.0, dtype=torch.bfloat16)]
    s = oz2.adamw_state(params, bits=8, master=True)
    assert s.exp_avg.shape == s.exp_avg_sq.shape == s.master.shape == (4 * 256,) and s.exp_avg_scale.shape == (4,)
    assert s.exp_avg.dtype == torch.float8_e4m3fn and s.exp_avg_sq.dtype == torch.uint8 and s.step.tolist() == [0, 0]
    want = torch.zeros(1024)
    want[:15], want[256:512], want[512:769] = 1.0, 2.0, 3.0
    assert torch.equal(s.master, want)
    s = oz2.adamw_state(params)
    assert s.exp_avg.dtype == s.exp_avg_sq.dtype == torch.float32 and s.exp_avg_scale is None and s.master is None
    with pytest.raises(TypeError):
        oz2.adamw_state([torch.ones(3)], master=True)
    with pytest.raises(ValueError):
        oz2.adamw_state(params, bits=16)
    with pytest.raises(ValueError):
        oz2.adamw_state([])


def test_e4m3_rounding_definition():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.normal(size=20000) * 10.0 ** rng.uniform(-4, 3, 20000), ref.E4M3[:127],
                        (ref.E4M3[:126] + ref.E4M3[1:127]) / 2]).astype(np.float32)
    x = x[np.abs(x) <= 448]  # torch's conversion does not saturate
    x = np.concatenate([x, -x])
    got = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(got, ref.to_e4m3(x))
    assert ref.to_e4m3(np.array([1e6, -1e6], np.float32)).tolist() == [126, 254]


def test_second_moment_rounding_keeps_the_mean():
    """Codes of one value over many draws: the mean is the value's to five deviations of it."""
    n = 1 << 14
    for x in (3e-9, 0.0007, 0.11, 0.73, 0.999):
        v = np.full(n, x, np.float32)
        v[::256] = 1.0  # the block's largest
        scale = np.full(n // 256, np.float32(255.0**-4))
        t = v / scale[0]
        ladder = ref.fourth(np.arange(256))
        k = np.searchsorted(ladder, t, side="right") - 1
        d = ref.draws(np.arange(n // 8), 1, 7)
        up = ((t - ladder[k]) * np.float32(65536) > d.astype(np.float32) * (ref.fourth(k + 1) - ladder[k])) | ((k == 0) & (t > 0))
        some = np.arange(n) % 256 != 0
        got = ref.fourth(np.minimum(k + up, 255))[some].astype(np.float64)
        if k[some].min() == 0:  # below the first step nothing becomes 0
            assert (got == 1).all()
            continue
        step = float(ref.fourth(k[some][:1] + 1)[0] - ladder[k[some][0]])
        assert abs(got.mean() - float(t[some][0])) <= 5 * step / 2 / got.size**0.5 + step * 2**-16
