"""The step operators against their definitions: rms_norm, token_logprobs and their gradients in 64 bits, adamw in 64
bits and, where its states have 8, to the bit.

Tolerances are error bounds, element by element.  u is half an ulp of the output type.  REL = 2^-17 bounds a row's norm in
32 bits relatively: a chain of at most 200 additions of positive terms (2^-24 each, halved by the root), a reciprocal
root of 2^-22 and a handful of products."""
import importlib.util
import math
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")
from tests import _steps_ref as ref  # noqa: E402
from tests._layers_ref import TINY, UNIT, act, assert_within  # noqa: E402
from tests._util import ROOT  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, F16, F32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
INF, NAN = float("inf"), float("nan")
REL = 2.0**-17
SEED = 0x1234567890ABCDEF


@pytest.fixture(scope="module")
def oz2():
    import __graft_entry__ as g

    g.build()
    import emulated_fp64_gemm_gb300 as m

    assert torch.cuda.is_available()
    yield m
    assert m.last_error() == 0


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(*shape, dtype=F32, seed=0, scale=1.0):
    return (torch.randn(*shape, generator=generator(seed + 17 * sum(shape)), device="cuda") * scale).to(dtype)


def strided(t, pad, shift):
    """t with rows `pad` elements longer apart and the first element `shift` elements into the storage."""
    rows, cols = t.shape
    store = torch.full((rows * (cols + pad) + shift + 8,), 77.0, device=t.device).to(t.dtype)
    view = store[shift:].as_strided((rows, cols), (cols + pad, 1))
    view.copy_(t)
    return view


def values(q):
    return torch.from_numpy(ref.E4M3).cuda()[q.view(torch.uint8).long()]


# ------------------------------------------------------------------ rms_norm
def check_norm(oz2, x, w, residual=None, eps=1e-6, quantize=False, block=None, **kw):
    dtype = x.dtype
    u, tiny = UNIT[dtype], TINY[dtype]
    want, s = ref.rms_norm(x.double(), w.double(), None if residual is None else residual.double(), eps)
    got = oz2.rms_norm(x, w, residual=residual, eps=eps, out_dtype=E4M3 if quantize else None, block=block, **kw)
    got = got if isinstance(got, tuple) else (got,)
    if residual is not None:
        assert_within(got[-1], s, (u + 2.0**-23) * s.abs() + tiny, "residual")
    if not quantize:
        assert_within(got[0], want, (REL + u * (1 + REL)) * want.abs() + tiny, "y")
        return got
    q, scale = got[:2]
    rows, cols = x.shape
    width = block or cols
    n = -(-cols // width)
    assert q.dtype == E4M3 and scale.shape == (rows, n)
    top = torch.nn.functional.pad(want, (0, n * width - cols)).view(rows, n, width).abs().amax(-1)
    assert_within(scale, top.clamp(min=1e-30) / 448, 2 * REL * top / 448 + 2.0**-22 * 1e-30, "scale")
    spread = scale.double().repeat_interleave(width, 1)[:, :cols]
    # half a step: 2^-4 of a normal value, half of 2^-9 below the least; and the norm's own error
    assert_within(values(q) * spread, want, (2.0**-4 + 4 * REL) * want.abs() + 2.0**-10 * spread * (1 + REL), "q")
    largest = torch.nn.functional.pad(values(q).abs(), (0, n * width - cols)).view(rows, n, width).amax(-1)
    assert bool((largest[top > 1e-29] == 448).all())  # a block's largest element is the type's
    return got


NORM_SIZES = [(1, 1), (3, 8), (5, 7), (2, 128), (9, 129), (4, 256), (33, 264), (17, 1000), (6, 1024), (7, 1032), (130, 2048), (11, 2051),
              (3, 4096), (5, 8192), (4, 8200), (3, 12345), (2, 16384), (2, 16392), (3, 20001), (1, 40000)]


@pytest.mark.parametrize("rows,cols", NORM_SIZES)
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_norm_over_sizes(oz2, rows, cols, dtype):
    x, r, w = normal(rows, cols, dtype=dtype), normal(rows, cols, dtype=dtype, seed=1), normal(cols, dtype=dtype, seed=2)
    check_norm(oz2, x, w)
    check_norm(oz2, x, w, r)
    for block in (None, 128):
        check_norm(oz2, x, w, r if cols % 3 else None, quantize=True, block=block)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", [200, 1001, 2048, 17000])
@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (3, 0), (0, 5), (16, 1), (4, 4)])
def test_norm_strides_and_alignment(oz2, dtype, cols, pad, shift):
    rows = 5
    x, r, w = normal(rows, cols, dtype=dtype), normal(rows, cols, dtype=dtype, seed=1), normal(cols, dtype=dtype, seed=2)
    xs, rs = strided(x, pad, shift), strided(r, pad + 8, shift)
    _, s = check_norm(oz2, xs, w, rs)
    out, res = strided(x, pad, shift), strided(r, pad, shift + 1)
    # (another alignment adds a row's squares in another order: the same bound, not the same bits)
    got = check_norm(oz2, xs, w, rs, out=out, residual_out=res)
    assert got[0] is out and got[1] is res and torch.equal(res, s)
    edge = out.as_strided((rows - 1, pad), (cols + pad, 1), out.storage_offset() + cols)
    assert bool((edge == 77).all())  # nothing is written between the rows
    q, scale, s8 = oz2.rms_norm(xs, w, residual=rs, out_dtype=E4M3, block=128)
    assert torch.equal(s8, s)
    # scales and codes do not depend on the layout by more than the sums' order
    q2, scale2 = oz2.rms_norm(x, w, residual=r, out_dtype=E4M3, block=128)[:2]
    assert_within(scale, scale2.double(), 2 * REL * scale2.double())
    out8 = torch.zeros(rows, cols + 13, dtype=torch.uint8, device="cuda").view(E4M3)[:, 5:5 + cols]
    got = oz2.rms_norm(xs, w, residual=rs, out_dtype=E4M3, block=128, out=out8)
    assert got[0] is out8 and torch.equal(out8.view(torch.uint8), q.view(torch.uint8)) and torch.equal(got[1], scale)
    # other layouts are copied
    assert torch.equal(oz2.rms_norm(x.t().contiguous().t(), w), oz2.rms_norm(x, w))


@pytest.mark.parametrize("cols", [96, 700, 2048, 20000])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_norm_in_place(oz2, cols, dtype):
    x, r, w = normal(6, cols, dtype=dtype), normal(6, cols, dtype=dtype, seed=1), normal(cols, dtype=dtype, seed=2)
    y, s = oz2.rms_norm(x, w, residual=r)
    a, b = x.clone(), r.clone()
    before = (a._version, b._version)
    got = oz2.rms_norm(a, w, residual=b, out=a, residual_out=b)
    assert got[0] is a and got[1] is b and torch.equal(a, y) and torch.equal(b, s)
    assert a._version > before[0] and b._version > before[1]
    a, b = x.clone(), r.clone()
    oz2.rms_norm(a, w, residual=b, out=b, residual_out=a)
    assert torch.equal(b, y) and torch.equal(a, s)
    b = r.clone()
    q, scale, _ = oz2.rms_norm(x, w, residual=b, out_dtype=E4M3, residual_out=b)
    assert torch.equal(b, s)


@pytest.mark.parametrize("cols", [64, 1000, 4096, 20000])
def test_norm_of_rows_whose_squares_leave_the_range(oz2, cols):
    # magnitudes from 1e-37 to 1e38; eps in reach of the small ones, and none
    size = 10.0 ** torch.tensor([-37.0, -30.0, -22.0, -15.0, -8.0, 0.0, 10.0, 19.0, 25.0, 36.0], device="cuda")
    for dtype in (F32, BF16):
        x = (normal(10, cols).clamp(-3, 3) * size[:, None]).to(dtype)
        w = normal(cols, dtype=dtype, seed=2)
        for eps in (0.0, 1e-30, 1e-6):
            check_norm(oz2, x, w, eps=eps)
        check_norm(oz2, x, w, eps=0.0, quantize=True)
        check_norm(oz2, x, w, eps=0.0, quantize=True, block=128)
        dy = normal(10, cols, dtype=dtype, seed=3)
        for eps in (0.0, 1e-6):
            check_norm_backward(oz2, dy, x[3:8], w, rows=slice(3, 8), eps=eps)
            check_norm_backward(oz2, dy, x, w, rows=slice(0, 10), eps=eps, weight=False)


@pytest.mark.parametrize("cols", [100, 1024, 2056, 18000])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_of_special_rows(oz2, cols, dtype):
    x, w = normal(6, cols, dtype=dtype), 1 + normal(cols, dtype=dtype, seed=2).abs()
    clean = oz2.rms_norm(x, w)
    bad = x.clone()
    bad[1] = 0
    bad[2, 3] = INF
    bad[3, 5] = NAN
    bad[4, cols - 1] = -INF
    got = oz2.rms_norm(bad, w)
    assert torch.equal(got[[0, 5]], clean[[0, 5]]) and not got[1].any() and bool(got[3].isnan().all())
    for row, at in ((2, 3), (4, cols - 1)):  # over an infinite norm finite elements are 0, infinity over infinity is not a number
        rest = torch.arange(cols, device="cuda") != at
        assert bool(got[row, at].isnan()) and not got[row, rest].any()
    for block in (None, 128):
        q, scale = oz2.rms_norm(bad, w, out_dtype=E4M3, block=block)
        q0, scale0 = oz2.rms_norm(x, w, out_dtype=E4M3, block=block)
        for row in (0, 5):
            assert torch.equal(q[row].view(torch.uint8), q0[row].view(torch.uint8)) and torch.equal(scale[row], scale0[row])
        assert not values(q)[1].any() and bool((scale[1].double() == float(np.float32(1e-30) * np.float32(1 / 448))).all())
        assert bool(values(q)[3].isnan().all()) and bool(scale[3].isnan().all())
        assert bool(scale[2, 0].isnan()) and bool(scale[4, -1].isnan())
    with pytest.raises(ValueError):
        oz2.rms_norm(bad, w, out_dtype=E4M3, block=64)


def check_norm_backward(oz2, dy, x, w, dres=None, rows=slice(None), eps=1e-6, weight=True, **kw):
    dy = dy[rows]
    u, tiny = UNIT[x.dtype], TINY[x.dtype]
    dx, dw, size, wsize = ref.rms_norm_backward(dy.double(), x.double(), w.double(), None if dres is None else dres.double(), eps)
    got, gotw = oz2.rms_norm_backward(dy, x, w, dresidual=dres, eps=eps, need_dweight=weight, **kw)
    assert_within(got, torch.where(dx.abs() > torch.finfo(x.dtype).max, INF * dx.sign(), dx),
                  4 * REL * size + u * (dx.abs() + 4 * REL * size) + tiny, "dx")
    if weight:
        assert_within(gotw, dw, 2 * REL * wsize + u * (dw.abs() + 2 * REL * wsize) + tiny, "dweight")
    else:
        assert gotw is None
    return got, gotw


@pytest.mark.parametrize("rows,cols", NORM_SIZES + [(700, 96), (1300, 520), (2500, 2048), (999, 4104), (40, 16400), (70, 17001)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_norm_backward_over_sizes(oz2, rows, cols, dtype):
    dy, x, d = (normal(rows, cols, dtype=dtype, seed=i) for i in range(3))
    w = normal(cols, dtype=dtype, seed=3)
    a = check_norm_backward(oz2, dy, x, w)
    b = check_norm_backward(oz2, dy, x, w, d)
    assert torch.equal(a[1], b[1])
    assert torch.equal(oz2.rms_norm_backward(dy, x, w, need_dweight=False)[0], a[0])
    # over what it reads
    for at in range(3):
        ts = [dy.clone(), x.clone(), d.clone()]
        got = oz2.rms_norm_backward(ts[0], ts[1], w, dresidual=ts[2], out=ts[at])
        assert got[0] is ts[at] and torch.equal(ts[at], b[0]) and torch.equal(got[1], b[1])


@pytest.mark.parametrize("pad,shift", [(8, 8), (3, 0), (0, 5), (9, 1)])
@pytest.mark.parametrize("dtype", [F16, F32])
def test_norm_backward_strides(oz2, dtype, pad, shift):
    for rows, cols in ((37, 1000), (5, 17000)):
        dy, x, d = (normal(rows, cols, dtype=dtype, seed=i) for i in range(3))
        w = normal(cols + 1, dtype=dtype, seed=3)[1:]
        out = strided(x, pad, shift)
        got, _ = check_norm_backward(oz2, strided(dy, pad, shift), strided(x, pad + 8, shift), w, strided(d, pad, shift + 1), out=out)
        assert got is out


def test_norm_gradient_against_differences(oz2):
    # in 32 bits, directions of the whole of x, residual and weight at once
    rows, cols, h = 4, 300, 2.0**-7
    x, r, w, dy = normal(rows, cols), normal(rows, cols, seed=1), normal(cols, seed=2), normal(rows, cols, seed=3)
    vx, vw, ds = normal(rows, cols, seed=4), normal(cols, seed=5), normal(rows, cols, seed=6)

    def value(t):
        y, s = oz2.rms_norm(x + t * vx, w + t * vw, residual=r)
        return float((y.double() * dy.double()).sum() + (s.double() * ds.double()).sum())

    s = oz2.rms_norm(x, w, residual=r)[1]
    dx, dw = oz2.rms_norm_backward(dy, s, w, dresidual=ds)
    slope = float((dx.double() * vx.double()).sum() + (dw.double() * vw.double()).sum())
    # the central difference is off by h^2 / 6 third derivatives (below 10 of this size) and by roundings over 2 h
    size = float((dx.abs() * vx.abs()).sum() + (dw.abs() * vw.abs()).sum())
    assert abs((value(h) - value(-h)) / (2 * h) - slope) <= size * (10 * h * h / 6 + 2.0**-22 / h)


def test_norm_empty(oz2):
    w = normal(16)
    x = torch.empty(0, 16, device="cuda")
    assert oz2.rms_norm(x, w).shape == (0, 16)
    q, scale = oz2.rms_norm(x, w, out_dtype=E4M3)
    assert q.shape == (0, 16) and scale.shape == (0, 1)
    dx, dw = oz2.rms_norm_backward(x, x, w)
    assert dx.shape == (0, 16) and not dw.any()
    none = torch.empty(3, 0, device="cuda")
    assert oz2.rms_norm(none, w[:0]).shape == (3, 0) and oz2.rms_norm_backward(none, none, w[:0])[0].shape == (3, 0)
    assert oz2.rms_norm(none, w[:0], out_dtype=E4M3, block=128)[1].shape == (3, 0)


@pytest.mark.parametrize("rows,cols,pad,shift", [(1, 9, 0, 1), (40, 5001, 0, 3), (700, 8, 1, 0), (650, 31, 0, 0), (1300, 777, 2, 5), (900, 2051, 0, 0),
                                                 (2000, 2041, 4, 7), (640, 4095, 0, 2), (5000, 130, 3, 1), (611, 8193, 0, 0), (620, 9999, 6, 6)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_norm_of_rows_off_boundaries(oz2, dtype, rows, cols, pad, shift):
    """All matrices' rows begin alike, within storages of NaN that no result may show and no call may change."""
    def within(t):
        store = torch.full((rows * (cols + pad) + shift + 16,), NAN, dtype=t.dtype, device="cuda")
        view = store[shift:].as_strided((rows, cols), (cols + pad, 1))
        view.copy_(t)
        return store, view

    def around(store, view):  # what is not the view's
        left = store.clone()
        left[shift:].as_strided((rows, cols), (cols + pad, 1)).fill_(0.0)
        return int(left.isnan().sum()) == store.numel() - rows * cols

    x, r, dy, d = (normal(rows, cols, dtype=dtype, seed=i) for i in range(4))
    w = within(normal(1, cols, dtype=dtype, seed=5).expand(rows, cols))[1][0]
    (_, xv), (_, rv), (_, dyv), (_, dv) = (within(t) for t in (x, r, dy, d))
    y_store, y = within(torch.zeros_like(x))
    s_store, s = within(torch.zeros_like(x))
    check_norm(oz2, xv, w, rv, out=y, residual_out=s)
    assert around(y_store, y) and around(s_store, s)
    check_norm(oz2, xv, w)
    check_norm(oz2, xv, w, rv, quantize=True)
    check_norm(oz2, xv, w, rv, quantize=True, block=128)
    q_store = torch.full((rows * (cols + pad) + shift + 16,), 0x7F, dtype=torch.uint8, device="cuda")
    q = q_store.view(E4M3)[shift:].as_strided((rows, cols), (cols + pad, 1))
    check_norm(oz2, xv, w, quantize=True, out=q)
    q_store[shift:].as_strided((rows, cols), (cols + pad, 1)).zero_()
    assert int((q_store == 0x7F).sum()) == q_store.numel() - rows * cols
    o_store, o = within(torch.zeros_like(x))
    got = check_norm_backward(oz2, dyv, xv, w, dv, out=o)
    assert around(o_store, o)
    plain = oz2.rms_norm_backward(dyv, xv, w, dresidual=dv)  # dx on boundaries, or as the inputs' rows are: one value
    check_norm_backward(oz2, dyv, xv, w)
    for into in range(3):
        ts = [within(t) for t in (dy, x, d)]
        over = oz2.rms_norm_backward(ts[0][1], ts[1][1], w, dresidual=ts[2][1], out=ts[into][1])
        assert torch.equal(over[0], got[0]) and torch.equal(over[1], got[1]) and around(*ts[into])
    assert_within(plain[0], got[0].double(), 2.0**-6 * got[0].double().abs() + 2.0**-7)
    xs, rs = within(x), within(r)
    z = oz2.rms_norm(xs[1], w, residual=rs[1], out=xs[1], residual_out=rs[1])
    assert torch.equal(z[0], y) and torch.equal(z[1], s) and around(*xs) and around(*rs)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", [300_000, 1_000_003])
def test_norm_of_the_longest_rows(oz2, dtype, cols):
    """A chain is of cols / 1024 squares: the norm is off by half of (cols / 1024 + 32) 2^-24, sums for dweight by their few rows."""
    rows, rel = 5, (cols / 1024 + 64) * 2.0**-24
    x, r, dy, ds, w = (normal(rows, cols, dtype=dtype, seed=i) for i in range(5))
    w = w[0]
    y, s = oz2.rms_norm(x, w, residual=r)
    want, ws = ref.rms_norm(x.double(), w.double(), r.double(), 1e-6)
    u = UNIT[dtype]
    assert_within(s, ws, (u + 2.0**-23) * ws.abs() + TINY[dtype])
    assert_within(y, want, (rel + u * (1 + rel)) * want.abs() + TINY[dtype])
    q, scale = oz2.rms_norm(x, w, residual=r, out_dtype=E4M3)[:2]
    top = want.abs().amax(-1, keepdim=True)
    assert_within(scale, top / 448, 2 * rel * top / 448)
    assert_within(values(q) * scale.double(), want, (2.0**-4 + 4 * rel) * want.abs() + 2.0**-10 * scale.double() * (1 + rel))
    dx, dw = oz2.rms_norm_backward(dy, x, w, dresidual=ds)
    wdx, wdw, size, wsize = ref.rms_norm_backward(dy.double(), x.double(), w.double(), ds.double(), 1e-6)
    # (the products' sum is not of one sign: off by that part of the sum of magnitudes, of which a row's x has its share)
    spread = (dy.double() * w.double() * x.double()).abs().mean(-1, keepdim=True) * x.double().abs() / (x.double()**2).mean(-1, keepdim=True).sqrt()**3
    assert_within(dx, wdx, 4 * rel * (size + spread) + u * (wdx.abs() + 4 * rel * (size + spread)) + TINY[dtype])
    assert_within(dw, wdw, 2 * rel * wsize + u * (wdw.abs() + 2 * rel * wsize) + TINY[dtype])


# ------------------------------------------------------------------ token_logprobs
def check_logprobs(oz2, logits, targets, temperature=1.0, top=0, ignore=-100, chains=512):
    """Against 64 bits.  A sum of V exponentials of 2^-21 each in 32 bits, about V / 512 in a chain (two per thread), is
    off by (V / 512 + 64) 2^-24 + 2^-21 relatively, and log p by the sizes of z - z_max and z_max times 2^-22 besides."""
    v = logits.shape[1]
    got = oz2.token_logprobs(logits, targets, temperature=temperature, top=top, entropy=True, ignore_index=ignore)
    z_max, log_sum, logp, entropy, every = ref.token_logprobs(logits, targets, temperature, ignore)
    rel = (v / chains + 64) * 2.0**-24 + 2.0**-21
    off = rel * (1 + log_sum) + 2.0**-22 * z_max.nan_to_num(0, 0, 0).abs()
    far = 2.0**-22
    assert_within(got.z_max, z_max, 2.0**-23 * z_max.nan_to_num(0, 0, 0).abs(), "z_max")
    assert_within(got.log_sum, log_sum, off, "log_sum")
    assert_within(got.logprobs, logp, off + far * logp.nan_to_num(0, 0, 0).abs(), "logprobs")
    assert_within(got.entropy, entropy, 4 * off * (1 + entropy), "entropy")
    if top:
        order = torch.sort(logits.float() + 0.0, dim=-1, descending=True, stable=True).indices[:, :top]
        assert torch.equal(got.top_ids, order)
        want = every.gather(1, order)
        assert_within(got.top_logprobs, want, off[:, None] + far * want.nan_to_num(0, 0, 0).abs(), "top")
    else:
        assert got.top_ids is None and got.top_logprobs is None
    less = oz2.token_logprobs(logits, targets, temperature=temperature, ignore_index=ignore)
    assert less.entropy is None
    assert torch.equal(less.z_max, got.z_max)
    assert_within(less.logprobs, got.logprobs.double(), 2 * off + 1e-37)
    return got


def some_targets(rows, vocab, seed=0):
    t = torch.randint(0, vocab, (rows,), generator=generator(seed), device="cuda")
    t[rows // 2::5] = -100
    return t


LOGIT_SIZES = [(1, 1), (3, 2), (2, 7), (5, 8), (4, 15), (1, 100), (7, 1000), (3, 4095), (2, 4096), (40, 8191), (1, 8192), (3, 32768), (2, 50021),
               (1, 131072), (20, 65537), (310, 20000), (160, 10001)]


@pytest.mark.parametrize("rows,vocab", LOGIT_SIZES)
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_logprobs_over_sizes(oz2, rows, vocab, dtype):
    logits = normal(rows, vocab, dtype=dtype, scale=3.0)
    for top, temperature in ((0, 1.0), (1, 0.7), (min(5, vocab), 1.0), (min(20, vocab), 2.0), (min(32, vocab), 1.0)):
        got = check_logprobs(oz2, logits, some_targets(rows, vocab), temperature, top)
        again = oz2.token_logprobs(logits, some_targets(rows, vocab), temperature=temperature, top=top, entropy=True)
        for a, b in zip(got, again):
            assert a is None and b is None or torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pad,shift", [(0, 1), (8, 0), (3, 5), (1, 7), (5, 2)])
def test_logprobs_strides(oz2, dtype, pad, shift):
    for rows, vocab in ((9, 1003), (4, 40000)):
        logits = normal(rows, vocab, dtype=dtype, scale=3.0)
        view = strided(logits, pad, shift)
        targets = torch.stack([some_targets(rows, vocab), some_targets(rows, vocab)], 1)[:, 0]
        a = check_logprobs(oz2, view, targets, top=8)
        b = oz2.token_logprobs(logits, targets.contiguous(), top=8)
        assert torch.equal(a.top_ids, b.top_ids)


def mask_rows(logits, value):
    """Rows with nothing masked, one token left, few, a block of neighbours, a comb, and none left."""
    rows, vocab = 8, logits.shape[1]
    keep = torch.zeros(rows, vocab, dtype=torch.bool, device="cuda")
    keep[0] = True
    keep[1, vocab // 2] = True
    keep[2, torch.randint(0, vocab, (5,), generator=generator(3), device="cuda")] = True
    keep[3, vocab // 3: vocab // 3 + min(2500, vocab // 2)] = True
    keep[4, ::max(1, vocab // 200)] = True
    keep[5, -1] = True
    keep[6, :40] = True
    return torch.where(keep, logits[:8], torch.full_like(logits[:8], value)), keep


@pytest.mark.parametrize("vocab", [9, 100, 5000, 33333, 131072])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("lowest", [False, True, -30000.0, -1e10, -3e25])
def test_logprobs_of_masked_rows(oz2, vocab, dtype, lowest):
    value = (torch.finfo(dtype).min if lowest is True or lowest < torch.finfo(dtype).min else lowest) if lowest else -INF
    logits, keep = mask_rows(normal(8, vocab, dtype=dtype, scale=3.0), value)
    targets = torch.arange(8, device="cuda") % vocab
    targets[1], targets[5] = vocab // 2, vocab - 1
    for top in (0, 1, min(20, vocab)):
        got = check_logprobs(oz2, logits, targets, top=top)
    # one token left: certain, with entropy 0; none left: nothing, or alike
    assert got.logprobs[1] == 0 and got.entropy[1] == 0 and got.logprobs[5] == 0
    if lowest:
        assert abs(float(got.log_sum[7]) - math.log(vocab)) <= 1e-5 * math.log(vocab) + 1e-6
    else:
        assert got.z_max[7] == -INF and got.logprobs[7] == -INF and got.log_sum[7] == 0 and got.entropy[7] == 0
        assert got.top_ids[7].tolist() == list(range(top)) and bool((got.top_logprobs[7] == -INF).all())


@pytest.mark.parametrize("vocab", [100, 5000, 60001])
def test_logprobs_ties(oz2, vocab):
    # a constant row, rows of few distinct values, zeros of both signs, and large values side by side in a few threads' reach
    logits = torch.zeros(7, vocab, device="cuda")
    logits[1] = torch.arange(vocab, device="cuda") % 3
    logits[2] = torch.where(torch.rand(vocab, generator=generator(1), device="cuda") < 0.5, 0.0, -0.0)
    logits[3] = -5.0
    logits[3, vocab // 2:] = 2.0
    logits[4] = normal(vocab).to(BF16).float()
    logits[5] = -1.0
    logits[5, 17:: 4096] = 1.0
    logits[6] = torch.arange(vocab, device="cuda").float() * 1e-3
    for dtype in (F32, BF16):
        for top in (1, 7, 32):
            check_logprobs(oz2, logits.to(dtype), torch.zeros(7, dtype=torch.int64, device="cuda"), top=top)


@pytest.mark.parametrize("vocab", [1030, 5003, 8191, 8192, 20011, 70000])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_logprobs_of_many_rows(oz2, vocab, dtype):
    # a warp or four to a row: what the tests above have in few rows, among ordinary ones
    rows = 8 * torch.cuda.get_device_properties(0).multi_processor_count + 3
    logits, columns = normal(rows, vocab, dtype=dtype, scale=3.0), torch.arange(vocab, device="cuda")
    for at, value in ((0, -INF), (8, torch.finfo(dtype).min), (16, -30000.0), (24, -1e10)):
        logits[at:at + 8] = mask_rows(logits[at:at + 8].clone(), value)[0]
    logits[32] = 0.0
    logits[33] = (columns % 3).to(dtype)
    logits[34, vocab // 2:] = 20.0
    for row, width in ((35, 8), (36, 32), (37, 100), (38, 248)):
        logits[row] = torch.where(columns % 1024 < width, 25 + torch.rand(vocab, generator=generator(row), device="cuda"), logits[row].float()).to(dtype)
    logits[39] = columns.to(dtype)
    logits[40] = (logits[40].float() * 100 + 1e6).to(dtype)
    logits[41, vocab - 1] = 60.0
    targets = some_targets(rows, vocab)
    targets[41] = vocab - 1
    for top in (0, 3, 32):
        check_logprobs(oz2, logits, targets, top=top, chains=64 if vocab < 8192 else 256)
    check_logprobs(oz2, strided(logits, 3, 1), targets, 0.7, top=9, chains=64 if vocab < 8192 else 256)


@pytest.mark.parametrize("rows,vocab,dtype", [(2, 3_000_001, F32), (90, 1_000_003, BF16), (330, 300_001, BF16), (1300, 150_001, F16)])
def test_logprobs_of_the_longest_rows(oz2, rows, vocab, dtype):
    # more passes of a thread than it notes apart: a cluster of eight, of two, eight warps, four
    logits = normal(rows, vocab, dtype=dtype, scale=3.0)
    logits[1, ::2] = -INF
    targets = some_targets(rows, vocab)
    got = oz2.token_logprobs(logits, targets, top=32, entropy=True)
    few = torch.tensor([0, 1, rows - 1], device="cuda")
    some = check_logprobs(oz2, logits[few], targets[few], top=32)
    assert torch.equal(got.top_ids[few], some.top_ids)
    rel = (vocab / 256 + 64) * 2.0**-24 + 2.0**-21  # of either one
    assert_within(got.logprobs[few], some.logprobs.double(), 2 * rel * (1 + some.log_sum.double()) + 2.0**-20 * some.logprobs.double().abs())
    d = oz2.token_logprobs_backward(torch.ones(rows, device="cuda"), logits, targets, got)
    p = torch.softmax(logits[few].double(), -1)
    onehot = torch.zeros_like(p).scatter_(1, targets[few].clamp(min=0)[:, None], 1.0) * (targets[few] >= 0)[:, None]
    want = torch.where((targets[few] >= 0)[:, None], onehot - p, 0.0)
    assert_within(d[few], want, (UNIT[dtype] + 2 * rel + 2.0**-18) * want.abs() + TINY[dtype])


@pytest.mark.parametrize("vocab", [40000, 262144])
def test_alternatives_in_few_threads(oz2, vocab):
    # thousands of distinct large logits in the reach of fewer threads than alternatives: more than there is room for
    logits = normal(24, vocab, scale=0.1)
    columns = torch.arange(vocab, device="cuda")
    for row, width in ((0, 32), (1, 100), (2, 8), (3, 248)):
        some = columns % 4096 < width
        logits[row] = torch.where(some, 5 + torch.rand(vocab, generator=generator(row), device="cuda"), logits[row])
    big = normal(400, vocab, scale=0.1, dtype=BF16)  # a block per row: threads with more elements each
    big[::7] = torch.where(columns % 4096 < 160, (5 + 3 * torch.rand(vocab, generator=generator(9), device="cuda")).to(BF16), big[::7])
    for x in (logits, big):
        for top in (20, 32):
            check_logprobs(oz2, x, torch.zeros(x.shape[0], dtype=torch.int64, device="cuda"), top=top)


@pytest.mark.parametrize("vocab", [10, 3001, 131072])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_logprobs_of_confident_rows(oz2, vocab, dtype):
    """log p of a token with almost all of the probability, and the entropy, keep their relative precision.

    With others of probability rho in all, log p = -log1p(rho): off by what rho is, a sum of exponentials of differences
    d (exact here, each exponential by 2^-21 and d's own rounding, |d| 2^-23): 2^-15 and (V / 512 + 64) 2^-24 in all."""
    gaps = torch.tensor([8.0, 12.0, 16.0, 20.0, 40.0, 60.0], device="cuda")
    at = torch.tensor([0, vocab // 2, vocab - 1, 3, 5, 1], device="cuda")
    logits = (normal(6, vocab) * 0.5).to(dtype).float()
    logits.scatter_(1, at[:, None], (gaps + math.log(vocab))[:, None].to(dtype).float())
    logits = logits.to(dtype)
    got = oz2.token_logprobs(logits, at, entropy=True, top=2)
    z = logits.double()
    d = z - z.gather(1, at[:, None])
    others = torch.exp(d).scatter(1, at[:, None], 0.0)
    rho = others.sum(1)
    rel = 2.0**-15 + (vocab / 512 + 64) * 2.0**-24
    assert_within(got.logprobs, -torch.log1p(rho), rel * rho)
    assert_within(got.log_sum, torch.log1p(rho), rel * rho)
    assert_within(got.top_logprobs[:, 0], -torch.log1p(rho), rel * rho)
    assert torch.equal(got.top_ids[:, 0], at)
    bent = -(others * d).sum(1)
    want = torch.log1p(rho) + bent / (1 + rho)
    assert_within(got.entropy, want, 2 * rel * want)


@pytest.mark.parametrize("vocab", [11, 5003, 70000])
@pytest.mark.parametrize("dtype", [F32, F16])
def test_logprobs_of_special_rows(oz2, vocab, dtype):
    x = normal(6, vocab, dtype=dtype)
    targets = torch.tensor([0, 1, 2, -100, vocab, -1], device="cuda")
    want = oz2.token_logprobs(x, targets, top=3, entropy=True)
    assert want.logprobs[3] == 0 and bool(want.logprobs[4:].isnan().all()) and bool(torch.isfinite(want.log_sum).all())
    bad = x.clone()
    bad[0, vocab - 1] = NAN
    bad[1, 4] = INF
    bad[3, 2] = NAN
    bad[3, 7] = INF
    got = oz2.token_logprobs(bad, targets, top=3, entropy=True)
    for a, b in zip(got, want):
        assert torch.equal(a[[2, 4, 5]].nan_to_num(7.0), b[[2, 4, 5]].nan_to_num(7.0))
        if a is not got.top_ids:
            assert bool(a[:2].isnan().all())
    assert got.logprobs[3] == 0 and bool(got.z_max[3].isnan()) and bool(got.entropy[3].isnan())
    assert got.top_ids[0, 0] == vocab - 1 and got.top_ids[1, 0] == 4 and got.top_ids[3, :2].tolist() == [2, 7]
    d = oz2.token_logprobs_backward(torch.ones(6, device="cuda"), bad, targets, got, dentropy=torch.ones(6, device="cuda"))
    assert bool(d[[0, 1, 3, 4, 5]].isnan().all()) and bool(torch.isfinite(d[2]).all())
    all_nan = torch.full((2, vocab), NAN, dtype=dtype, device="cuda")
    assert oz2.token_logprobs(all_nan, targets[:2], top=3).top_ids.tolist() == [[0, 1, 2]] * 2
    # another number for what is ignored
    one = oz2.token_logprobs(x, targets, ignore_index=1)
    assert one.logprobs[1] == 0 and bool(one.logprobs[3].isnan())


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shift", [300.0, -5e3, 6e4, 1e6, -3e7, 1e12])
def test_logprobs_of_logits_far_from_zero(oz2, dtype, shift):
    if abs(shift) > torch.finfo(dtype).max:
        return
    # (their differences are multiples of the type's steps there, some of them of an ordinary size)
    step = abs(shift) * torch.finfo(dtype).eps
    logits = (normal(6, 5000, scale=3.0) * max(1.0, step) + shift).to(dtype)
    targets = logits.float().argmax(-1)
    targets[3:] = 7
    check_logprobs(oz2, logits, targets, top=5)
    if shift < 0:  # beside ordinary ones nothing is left of them
        logits[:, 4000:] = normal(6, 1000, dtype=dtype)
        check_logprobs(oz2, logits, torch.full_like(targets, 4321), top=5)
    check_logprobs_backward(oz2, logits, targets)


def test_logprobs_temperatures(oz2):
    x = normal(5, 3000, scale=4.0)
    for temperature in (1e-3, 0.1, 30.0, 1e6):
        check_logprobs(oz2, x, some_targets(5, 3000), temperature, top=4)
    # so high that masked logits alone leave the softmax, however low the others are; so low that one logit is left
    for dtype in (F32, BF16, F16):
        logits, _ = mask_rows(normal(8, 9000, dtype=dtype, scale=3.0), -INF)
        targets = torch.tensor([0, 4500, 0, 3000, 0, 8999, 1, 0], device="cuda")
        check_logprobs(oz2, logits, targets, 1e-20, top=3)
        logits[0, ::3] = torch.finfo(dtype).min
        logits[6] = torch.finfo(dtype).min
        logits[6, 7] = -INF
        for temperature in (1e9, 1e30):
            check_logprobs(oz2, logits, targets, temperature, top=3)
    # z passes the 32-bit range: where it falls to -inf it is masked, a row of nothing else has no distribution
    low = torch.full((2, 100), -3e38, device="cuda")
    low[1, 5] = 1.0
    got = oz2.token_logprobs(low, torch.tensor([5, 5], device="cuda"), temperature=0.5, entropy=True)
    assert got.z_max.tolist() == [-INF, 2.0] and got.logprobs.tolist() == [-INF, 0.0] and got.entropy.tolist() == [0.0, 0.0]


def check_logprobs_backward(oz2, logits, targets, temperature=1.0, entropy=True, ignore=-100, **kw):
    """p is off by what log p is: (V / 512 + 64) 2^-24 + 2^-20 and the sizes of z_max and z - z_max times 2^-22."""
    rows, vocab = logits.shape
    u, tiny = UNIT[logits.dtype], TINY[logits.dtype]
    g, h = normal(rows, seed=5), normal(rows, seed=6) if entropy else None
    saved = oz2.token_logprobs(logits, targets, temperature=temperature, entropy=entropy, ignore_index=ignore)
    got = oz2.token_logprobs_backward(g, logits, targets, saved, dentropy=h, temperature=temperature, ignore_index=ignore, **kw)
    z_max, log_sum, _, ent, logp = ref.token_logprobs(logits, targets, temperature, ignore)
    p = torch.where((z_max > -INF)[:, None], torch.exp(logp), 0.0)
    known = (targets != ignore) & (z_max > -INF)
    gd = torch.where(known, g.double(), 0.0)[:, None]
    onehot = torch.zeros_like(p).scatter_(1, torch.where(targets == ignore, 0, targets)[:, None], 1.0)
    # 1 - p of the target is formed without cancellation, as -expm1(log p)
    at_target = -torch.expm1(torch.where(torch.isfinite(logp), logp, -1e300))
    base = torch.where((onehot > 0) & known[:, None], gd * at_target, -gd * p)
    near = logp.clamp(min=-200)
    bend = h.double()[:, None] * p * (near + ent[:, None]) if entropy else torch.zeros_like(p)
    # log p below -100 has no part in 32 bits
    rel = (vocab / 512 + 64) * 2.0**-24 + 2.0**-20 + 2.0**-22 * (z_max.abs().clamp(max=1e4)[:, None].nan_to_num(0) + near.abs().clamp(max=200))
    size = gd.abs() * torch.where(onehot > 0, at_target.abs() + 2.0**-20 * p, p)
    if entropy:
        size = size + 2 * h.double().abs()[:, None] * p * (1 + near.abs() + ent[:, None])
    err = (2 * rel * size + 2.0**-120) / temperature
    want = (base - bend) / temperature
    assert_within(got, want, err + u * (want.abs() + err) + tiny, "dlogits")
    return got, saved, g, h


@pytest.mark.parametrize("rows,vocab", [s for s in LOGIT_SIZES if s[0] * s[1] <= 10**7])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_logprobs_backward_over_sizes(oz2, rows, vocab, dtype):
    logits, targets = normal(rows, vocab, dtype=dtype, scale=3.0), some_targets(rows, vocab)
    for temperature, entropy in ((1.0, True), (0.7, False), (1.3, True)):
        got, saved, g, h = check_logprobs_backward(oz2, logits, targets, temperature, entropy)
    over = logits.clone()
    version = over._version
    d = oz2.token_logprobs_backward(g, over, targets, saved, dentropy=h, temperature=temperature, out=over)
    assert d is over and torch.equal(over, got) and over._version > version


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pad,shift", [(0, 1), (8, 0), (3, 5)])
def test_logprobs_backward_strides(oz2, dtype, pad, shift):
    rows, vocab = 5, 9001
    logits, targets = normal(rows, vocab, dtype=dtype, scale=3.0), some_targets(rows, vocab)
    want, *_ = check_logprobs_backward(oz2, logits, targets)
    got, *_ = check_logprobs_backward(oz2, strided(logits, pad, shift), targets)
    assert_within(got, want.double(), 1e-4 * want.double().abs() + 2 * UNIT[dtype] * want.double().abs() + 1e-30)
    for p, s in ((pad, shift), (pad + 3, shift + 2)):
        out = strided(logits, p, s)
        check_logprobs_backward(oz2, strided(logits, pad, shift), targets, out=out)
        edge = out.as_strided((rows - 1, p), (vocab + p, 1), out.storage_offset() + vocab)
        assert bool((edge == 77).all())


@pytest.mark.parametrize("vocab", [9, 5000, 33333])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lowest", [False, True, -30000.0, -1e10, -3e25])
def test_logprobs_backward_of_masked_rows(oz2, vocab, dtype, lowest):
    value = (torch.finfo(dtype).min if lowest is True or lowest < torch.finfo(dtype).min else lowest) if lowest else -INF
    logits, keep = mask_rows(normal(8, vocab, dtype=dtype, scale=3.0), value)
    targets = torch.arange(8, device="cuda") % vocab
    targets[1], targets[4] = vocab // 2, -100
    for entropy in (False, True):
        got, *_ = check_logprobs_backward(oz2, logits, targets, entropy=entropy)
        if not lowest:
            others = ~keep.scatter(1, targets.clamp(min=0)[:, None], True)
            assert not got[others].any() and not got[7].any()


def test_logprobs_gradient_against_differences(oz2):
    rows, vocab, h = 6, 1000, 2.0**-6
    x, v = normal(rows, vocab, scale=2.0), normal(rows, vocab, seed=1)
    targets = some_targets(rows, vocab)
    g, e = normal(rows, seed=2), normal(rows, seed=3)

    def value(t):
        r = oz2.token_logprobs(x + t * v, targets, temperature=0.8, entropy=True)
        return float((r.logprobs.double() * g.double()).sum() + (r.entropy.double() * e.double()).sum())

    saved = oz2.token_logprobs(x, targets, temperature=0.8, entropy=True)
    d = oz2.token_logprobs_backward(g, x, targets, saved, dentropy=e, temperature=0.8)
    slope, size = float((d.double() * v.double()).sum()), float((d.double() * v.double()).abs().sum())
    # third derivatives of log p and the entropy along v are below 100 times |g| and |e|; values below 10 have roundings of 2^-20
    bound = h * h / 6 * 100 * float(g.abs().sum() + e.abs().sum()) + rows * 2.0**-20 * 4 / h
    assert abs((value(h) - value(-h)) / (2 * h) - slope) <= bound and bound < 0.5 * size


def test_logprobs_empty(oz2):
    x, t = torch.empty(0, 50, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    got = oz2.token_logprobs(x, t, top=3, entropy=True)
    assert got.logprobs.shape == got.entropy.shape == (0,) and got.top_ids.shape == (0, 3)
    assert oz2.token_logprobs_backward(got.logprobs, x, t, got).shape == (0, 50)
    with pytest.raises(ValueError):
        oz2.token_logprobs(torch.empty(2, 0, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda"))


# ------------------------------------------------------------------ adamw
OPTIONS = dict(lr=3e-3, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)


def tensors(sizes, dtype, grad_dtype, seed=0, shift=0):
    """Parameters and gradients of these sizes, each `shift` elements into a storage of its own."""
    params, grads = [], []
    for i, n in enumerate(sizes):
        shape = (n // 8, 8) if n and n % 8 == 0 else (n,)
        for into, t, scale, s in ((params, dtype, 0.1, 2 * i), (grads, grad_dtype, 0.01, 2 * i + 1)):
            store = normal(n + shift, dtype=t, scale=scale, seed=seed + s)
            into.append(store[shift:].view(shape))
    return params, grads


def offsets(sizes):
    at = [0]
    for n in sizes:
        at.append(at[-1] + -(-n // 256) * 256)
    return at


def check_step(oz2, params, grads, state, grad_scale=1.0, **kw):
    """One step against 64 bits, and 8-bit states against single roundings."""
    o = {**OPTIONS, **kw}
    t = int(state.step[0]) + 1
    sizes = [p.numel() for p in params]
    eight = state.exp_avg_scale is not None
    before = [None if s is None else s.clone() for s in state]
    old = [p.clone() for p in params]
    oz2.adamw(params, grads, state, grad_scale=grad_scale, **o)
    assert state.step.tolist() == [t, 0]
    b1, b2 = o["betas"]
    m0, v0 = before[1], before[2]
    if eight:
        m0 = values(m0) * before[3].double().repeat_interleave(256)
        v0 = v0.double()**4 * before[4].double().repeat_interleave(256)
    lr = float(o["lr"])
    for p, p0, g, n, at in zip(params, old, grads, sizes, offsets(sizes)):
        here = slice(at, at + n)
        gd = g.double().flatten() * float(grad_scale)
        m, v = b1 * m0[here].double() + (1 - b1) * gd, b2 * v0[here].double() + (1 - b2) * gd * gd
        m_size = (b1 * m0[here].double()).abs() + ((1 - b1) * gd).abs()
        w0 = (p0 if state.master is None else before[5][here]).double().flatten()
        root = torch.sqrt(v / (1 - b2**t)) + o["eps"]
        want = w0 * (1 - lr * o["weight_decay"]) - lr * m / (1 - b1**t) / root
        # 32 bits: a few roundings of 2^-24 of each term, the approximate root and reciprocal of 2^-22, 1 - b^t of 2^-22
        err = 2.0**-22 * w0.abs() + 2.0**-19 * lr * m_size / (1 - b1**t) / root
        u, tiny = UNIT[p.dtype], TINY[p.dtype]
        if state.master is not None:
            assert_within(state.master[here], want, err, "master")
            assert torch.equal(p.flatten(), state.master[here].to(p.dtype))
        else:
            assert_within(p.flatten(), want, err + u * (want.abs() + err) + tiny, "param")
        if not eight:
            assert_within(state.exp_avg[here], m, 2.0**-22 * m_size + 2.0**-148, "exp_avg")
            assert_within(state.exp_avg_sq[here], v, 2.0**-22 * v + 2.0**-148, "exp_avg_sq")
            continue
        blocks = slice(at // 256, at // 256 + -(-n // 256))
        whole = slice(at, at + -(-n // 256) * 256)
        inside = np.arange(whole.stop - at) < n
        g32 = np.zeros(inside.size, np.float32)
        g32[:n] = g.float().flatten().cpu().numpy() * np.float32(float(grad_scale))
        codes = [np.where(inside, s[whole].view(torch.uint8).cpu().numpy(), 0) for s in before[1:3]]
        scales = [s[blocks].cpu().numpy() for s in before[3:5]]
        _, _, mq, vq, ms, vs = ref.adamw_moments8(*codes, *scales, g32, b1, b2, t, o.get("seed", 0), at // 8)
        assert np.array_equal(state.exp_avg_scale[blocks].cpu().numpy(), ms)
        assert np.array_equal(state.exp_avg_sq_scale[blocks].cpu().numpy(), vs)
        assert np.array_equal(state.exp_avg[here].view(torch.uint8).cpu().numpy(), mq[inside])
        assert np.array_equal(state.exp_avg_sq[here].cpu().numpy(), vq[inside])
        if inside.sum() < inside.size:  # the gap is not changed
            gap = slice(at + n, whole.stop)
            assert torch.equal(state.exp_avg[gap].view(torch.uint8), before[1][gap].view(torch.uint8))
            assert torch.equal(state.exp_avg_sq[gap], before[2][gap])


KINDS = [(F32, F32, False), (BF16, BF16, False), (F16, F16, False), (BF16, F32, True), (F16, F16, True), (BF16, BF16, True), (BF16, F32, False)]


@pytest.mark.parametrize("dtype,grad_dtype,master", KINDS)
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("sizes", [[1], [256], [7, 0, 255, 257, 1000], [0, 0, 4096, 12344, 0], [300] * 30, [3, 70000, 512]])
def test_adamw_over_sizes(oz2, dtype, grad_dtype, master, bits, sizes):
    for shift in (0, 3):
        params, _ = tensors(sizes, dtype, grad_dtype, shift=shift)
        state = oz2.adamw_state(params, bits=bits, master=master)
        for step in range(4):
            grads = tensors(sizes, dtype, grad_dtype, seed=1000 * step, shift=shift)[1]
            check_step(oz2, params, grads, state, seed=SEED)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_of_many_tensors(oz2, bits):
    # more than one launch holds, empty ones among them and at the end; and enough elements for the longer form
    for sizes in ([1 + i % 600 if i % 7 else 0 for i in range(2000)] + [0, 0], [33_000_003, 5, 60_000_000]):
        params, grads = tensors(sizes, BF16, BF16)
        state = oz2.adamw_state(params, bits=bits)
        flat = torch.cat([p.flatten() for p in params])
        oz2.adamw(params, grads, state, seed=1, **OPTIONS)
        assert state.step.tolist() == [1, 0]
        # after a first step m' is the gradient and v' its square
        p0, g0 = flat.double(), torch.cat([g.flatten() for g in grads]).double()
        want = p0 * (1 - OPTIONS["lr"] * 0.1) - OPTIONS["lr"] * g0 / (g0.abs() + OPTIONS["eps"])
        assert_within(torch.cat([p.flatten() for p in params]), want, 2.0**-8 * want.abs() + 2.0**-18 * OPTIONS["lr"])
        for i in range(0, len(sizes), 97):  # its states are each tensor's own
            at = offsets(sizes)[i]
            assert not sizes[i] or bool(state.exp_avg[at:at + sizes[i]].float().abs().sum() > 0)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_scales_and_numbers_in_memory(oz2, bits):
    sizes = [1000, 77]
    runs = []
    for where in (False, True):
        params, grads = tensors(sizes, F32, F32)
        state = oz2.adamw_state(params, bits=bits)
        for lr, scale in ((1e-3, 0.5), (2e-3, 0.25)):
            number = (lambda v: torch.tensor([v], device="cuda")) if where else float  # noqa: E731
            check_step(oz2, params, grads, state, grad_scale=number(scale), lr=number(lr), seed=3)
        runs.append(params)
    for a, b in zip(*runs):
        assert torch.equal(a, b)


def test_adamw_of_extreme_gradients(oz2):
    # rows of zeros, gradients at the ends of the range, one infinity
    params, grads = tensors([1024, 512], F32, F32)
    grads[0].view(-1)[:256] = 0
    grads[0].view(-1)[256:512] *= 1e-24
    grads[0].view(-1)[512:768] *= 1e20
    for bits in (32, 8):
        p = [t.clone() for t in params]
        state = oz2.adamw_state(p, bits=bits)
        for _ in range(3):
            check_step(oz2, p, grads, state, seed=5)
        bad = [g.clone() for g in grads]
        bad[1].view(-1)[300] = INF
        oz2.adamw(p, bad, state, seed=5, **OPTIONS)
        fine = torch.isfinite(p[1].flatten())
        assert bool(torch.isfinite(p[0]).all()) and int((~fine).sum()) == 1
        m = state.exp_avg[1024:].float() if bits == 32 else values(state.exp_avg[1024:]) * state.exp_avg_scale[4:].double().repeat_interleave(256)
        lost = ~torch.isfinite(m)
        assert bool(lost[300]) and not lost[:256].any() and int(lost.sum()) <= (1 if bits == 32 else 256)


def test_second_moment_follows_its_mean_in_8_bits(oz2):
    """Constant gradients of many sizes: v tends to g^2 although each step changes it by far less than a step of its code."""
    n, steps, b2 = 1 << 16, 600, 0.99
    size = torch.linspace(0.3, 1.0, n, device="cuda")[torch.randperm(n, generator=generator(1), device="cuda")]
    params, grads = [torch.zeros(n, device="cuda")], [size.clone()]
    state = oz2.adamw_state(params, bits=8)
    for _ in range(steps):
        oz2.adamw(params, grads, state, lr=0.0, betas=(0.9, b2), seed=2)
    v = state.exp_avg_sq.double()**4 * state.exp_avg_sq_scale.double().repeat_interleave(256)
    ratio = v / size.double()**2
    # a step's rounding has a deviation of at most half a code's step (below 4 / 255 / 0.3^0.5 = 3 % of v), kept over
    # 1 / (1 - b2^2) = 50 steps: 0.5 * 0.03 * 50^0.5 = 11 %; the mean of 2^16 is within 5 * 11 % / 256 and what 600 steps leave
    assert abs(float(ratio.mean()) - 1) <= 5 * 0.11 / 256 + 2 * b2**steps
    assert float((ratio - 1).abs().max()) <= 6 * 0.11


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype,master", [(F32, False), (BF16, True)])
def test_adamw_states_within_a_storage(oz2, bits, dtype, master):
    # parameters and states that begin anywhere
    params, grads = tensors([1000, 77, 513], dtype, dtype, shift=3)
    state = oz2.adamw_state(params, bits=bits, master=master)
    by = [1, 3 if bits == 32 else 8, 5 if bits == 32 else 16, 1, 3, 7]
    moved = [None if t is None else torch.zeros(t.numel() + n + 4, dtype=t.dtype, device="cuda")[n:n + t.numel()] for t, n in zip(state, by)]
    if master:
        moved[5].copy_(state.master)
    state = oz2.AdamWState(*moved)
    for _ in range(2):
        check_step(oz2, params, grads, state, seed=4)
    if bits == 8:
        with pytest.raises(oz2.Ozaki2Error):
            oz2.adamw(params, grads, state._replace(exp_avg=torch.zeros(state.exp_avg.numel() + 1, dtype=E4M3, device="cuda")[1:]), **OPTIONS)
        assert state.step.tolist() == [2, 0]


def test_adamw_refusals(oz2):
    params, grads = tensors([64, 32], BF16, BF16)
    state = oz2.adamw_state(params)
    ok = dict(lr=1e-3)
    for p, g, s in (([], [], state), (params, grads[:1], state), (params[::-1], grads, state), (params, grads, state._replace(step=state.step[:1])),
                    (params, grads, state._replace(exp_avg_scale=state.exp_avg)), ([params[0].t(), params[1]], [grads[0].t(), grads[1]], state),
                    (params, grads, state._replace(exp_avg=state.exp_avg[:-1])), ([t.cpu() for t in params], grads, state)):
        with pytest.raises(ValueError):
            oz2.adamw(p, g, s, **ok)
    with pytest.raises(TypeError):
        oz2.adamw([params[0], params[1].float()], grads, state, **ok)
    with pytest.raises(TypeError):
        oz2.adamw(params, [g.half() for g in grads], state, **ok)
    with pytest.raises(oz2.Ozaki2Error):
        oz2.adamw([params[0], params[0]], [grads[0], grads[0]], oz2.adamw_state([params[0], params[0]]), **ok)
    with pytest.raises(oz2.Ozaki2Error):
        oz2.adamw(params, grads, state, lr=1e-3, betas=(0.9, 1.0))
    assert state.step.tolist() == [0, 0]


# ------------------------------------------------------------------ streams, graphs, autograd, size
def test_streams_and_graphs(oz2):
    rows, dim, vocab = 48, 512, 4100
    x, r, w = normal(rows, dim, dtype=BF16), normal(rows, dim, dtype=BF16, seed=1), normal(dim, dtype=BF16, seed=2)
    logits, targets = normal(rows, vocab, dtype=BF16, scale=2.0), some_targets(rows, vocab)
    dy, g = normal(rows, dim, dtype=BF16, seed=3), normal(rows, seed=4)
    params, grads = tensors([4000, 300], BF16, BF16)

    def calls(p, state, stream=None):
        a = oz2.rms_norm(x, w, residual=r, stream=stream)
        q = oz2.rms_norm(x, w, out_dtype=E4M3, block=128, stream=stream)
        b = oz2.rms_norm_backward(dy, x, w, dresidual=r, stream=stream)
        c = oz2.token_logprobs(logits, targets, top=6, entropy=True, stream=stream)
        d = oz2.token_logprobs_backward(g, logits, targets, c, dentropy=g, stream=stream)
        oz2.adamw(p, grads, state, seed=9, stream=stream, **OPTIONS)
        return [*a, q[0].view(torch.uint8), q[1], *b, *c, d]

    def fresh():
        p = [t.clone() for t in params]
        return p, oz2.adamw_state(p, bits=8, master=True)

    p, state = fresh()
    want = [calls(p, state) for _ in range(3)][0]
    wanted = [t.clone() for t in (*p, *state)]
    side = torch.cuda.Stream()
    p, state = fresh()
    side.wait_stream(torch.cuda.current_stream())
    got = [calls(p, state, side) for _ in range(3)][0]
    side.synchronize()
    for a, b in zip([*got, *p, *state], [*want, *wanted]):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    # a captured step counts on with every replay
    p, state = fresh()
    calls(*fresh())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = calls(p, state)
    assert state.step.tolist() == [0, 0]
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip([*got, *p, *state], [*want, *wanted]):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_calls_at_once(oz2):
    """Two streams' calls, two graphs captured on them, and two host threads: each as if it were alone."""
    import threading

    rows, dim, vocab = 3000, 2048, 20001
    sets = []
    for seed in (0, 100):
        x, dy, w = normal(rows, dim, dtype=BF16, seed=seed), normal(rows, dim, dtype=BF16, seed=seed + 1), normal(dim, dtype=BF16, seed=seed + 2)
        sets.append((x, dy, w, normal(1200, vocab, dtype=BF16, seed=seed + 3), some_targets(1200, vocab, seed), normal(1200, seed=seed + 4),
                     *tensors([500_000, 33, 70_001], BF16, BF16, seed=seed)))

    def calls(data, stream=None):
        x, dy, w, logits, targets, g, params, grads = data
        p = [t.clone() for t in params]
        state = oz2.adamw_state(p, bits=8)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        out = []
        for _ in range(3):
            out += oz2.rms_norm_backward(dy, x, w, stream=stream)
            saved = oz2.token_logprobs(logits, targets, top=4, stream=stream)
            out += [saved.logprobs, saved.top_ids, oz2.token_logprobs_backward(g, logits, targets, saved, stream=stream)]
            oz2.adamw(p, grads, state, seed=2, stream=stream, **OPTIONS)
        return [*out, *p, *(t for t in state if t is not None)]

    def same(got):
        torch.cuda.synchronize()
        for a, b in zip(got, wanted):
            for s, t in zip(a, b):
                assert torch.equal(s.view(torch.uint8), t.view(torch.uint8))

    wanted = [calls(data) for data in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    same([calls(data, stream) for data, stream in zip(sets, streams)])

    got = [None, None]

    def thread(i):
        with torch.cuda.stream(streams[i]):
            got[i] = calls(sets[i])

    torch.cuda.synchronize()
    threads = [threading.Thread(target=thread, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    same(got)

    graphs, got = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for graph, stream, data in zip(graphs, streams, sets):
        with torch.cuda.graph(graph, stream=stream):
            got.append(calls(data))
    for _ in range(2):  # (a replay makes its own copies of the parameters and states)
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        same(got)


def test_autograd_notices_the_step(oz2):
    w = normal(64).requires_grad_(True)
    loss = (w * w).sum()
    state = oz2.adamw_state([w])
    version = w._version
    oz2.adamw([w], [torch.ones_like(w)], state, lr=0.1)
    assert w._version > version
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_more_than_2_31_elements(oz2):
    # rows whose offsets pass 31 and 32 bits, in every operator
    cols = 4096
    rows = (1 << 32) // cols + 40
    x = torch.zeros(rows, cols, dtype=BF16, device="cuda")
    few = normal(7, cols, dtype=BF16)
    at = torch.tensor([0, 1, (1 << 31) // cols - 1, (1 << 31) // cols, (1 << 32) // cols - 1, (1 << 32) // cols, rows - 1], device="cuda")
    x[at] = few
    w = normal(cols, dtype=BF16, seed=1)
    y = oz2.rms_norm(x, w)
    assert torch.equal(y[at], oz2.rms_norm(few, w)) and not y[2].any()
    targets = torch.zeros(rows, dtype=torch.int64, device="cuda")
    a, b = oz2.token_logprobs(x, targets, top=3, entropy=True), oz2.token_logprobs(few, targets[:7], top=3, entropy=True)
    assert torch.equal(a.top_ids[at], b.top_ids)
    assert_within(a.logprobs[at], b.logprobs.double(), 1e-5 * b.logprobs.double().abs())
    assert_within(a.logprobs[2:3], torch.tensor([-math.log(cols)], dtype=torch.float64, device="cuda"), 1e-5)
    del y
    g = torch.ones(rows, device="cuda")
    d = oz2.token_logprobs_backward(g, x, targets, a)
    want = oz2.token_logprobs_backward(g[:7], few, targets[:7], b)
    assert_within(d[at], want.double(), 2.0**-7 * want.double().abs() + 1e-9)
    d.zero_()
    d[at] = few
    dx, dw = oz2.rms_norm_backward(d, x, w, out=d)
    small, dws = oz2.rms_norm_backward(few, few, w)
    assert torch.equal(dx[at], small) and not dx[2].any()
    assert_within(dw, dws.double(), 2.0**-7 * dws.double().abs() + 2.0**-16)
    del d, dx
    grads = [x.view(-1)]
    params = [torch.zeros(rows * cols, dtype=BF16, device="cuda")]
    state = oz2.adamw_state(params, bits=8)
    oz2.adamw(params, grads, state, lr=0.125, weight_decay=0.0, eps=1e-12)
    got = params[0].view(rows, cols)
    assert_within(got[at], -0.125 * few.double().sign(), 2.0**-8 * 0.125)
    assert not got[2].any()


# ------------------------------------------------------------------ together
def test_language_model_example(oz2):
    """The example's step: its loss and gradients against 64-bit autograd of the same model, its updates, and its 8-bit norm."""
    spec = importlib.util.spec_from_file_location("language_model", os.path.join(ROOT, "examples", "language_model.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    model = ex.Model(vocab=1003, dim=256, hidden=768, layers=2)
    ids = torch.randint(0, 1003, (96,), generator=generator(1), device="cuda")
    targets = ids.roll(-1).clone()
    targets[::9] = -100
    loss, grads = model.loss_and_gradients(ids, targets, bonus=0.01)

    w = {n: v.detach().double().requires_grad_(True) for n, v in model.w.items()}
    s, h = w["embed"][ids], None
    for i in range(2):
        y, s = ref.rms_norm(s, w[f"norm{i}"], h, 1e-6)
        h = act(y @ w[f"up{i}"].t() + w[f"up{i}_b"], "silu") @ w[f"down{i}"].t() + w[f"down{i}_b"]
    y, s = ref.rms_norm(h, w["norm"], s, 1e-6)
    _, _, logp, entropy, _ = ref.token_logprobs(y @ w["head"].t(), targets, 1.0, -100)
    want = -(logp.sum() + 0.01 * entropy.sum()) / len(ids)
    exact = torch.autograd.grad(want, list(w.values()))
    assert abs(float(loss) - float(want.detach())) <= 0.01 * abs(float(want.detach()))
    # a chain of about ten bfloat16 roundings of 2^-9 each: 3 % of the norm is six times their sum
    for (name, got), e in zip(grads.items(), exact):
        assert float((got.double() - e).norm()) <= 0.03 * float(e.norm()), name
    before = {n: v.clone() for n, v in model.w.items()}
    for bits in (32, 8):
        model.train(ids, targets, steps=2, bits=bits)
    assert all(not torch.equal(before[n], v) and bool(torch.isfinite(v).all()) for n, v in model.w.items())
    ids, logprobs = model.alternatives(ids[:3], top=4)
    assert ids.shape == logprobs.shape == (3, 4) and bool((logprobs[:, :-1] >= logprobs[:, 1:]).all())


# ------------------------------------------------------------------ refusals
def test_refusals(oz2):
    x, w, t = normal(4, 16), normal(16), torch.zeros(4, dtype=torch.int64, device="cuda")
    saved = oz2.token_logprobs(x, t)
    g = torch.ones(4, device="cuda")
    for f in (lambda: oz2.rms_norm(x, w[:8]), lambda: oz2.rms_norm(x[0], w), lambda: oz2.rms_norm(x, w, residual=x[:2]),
              lambda: oz2.rms_norm(x, w, residual_out=x), lambda: oz2.rms_norm(x, w, block=128),
              lambda: oz2.rms_norm(x, w, residual=x, out=x, residual_out=x), lambda: oz2.rms_norm(x, w, out=x.t()),
              lambda: oz2.rms_norm(x.cpu(), w), lambda: oz2.rms_norm(x, w.cpu()), lambda: oz2.rms_norm_backward(x, x[:2], w),
              lambda: oz2.token_logprobs(x, t[:3]), lambda: oz2.token_logprobs(x, t, top=17), lambda: oz2.token_logprobs(x, t, top=-1),
              lambda: oz2.token_logprobs(x, t, temperature=0.0), lambda: oz2.token_logprobs(x, t, temperature=NAN),
              lambda: oz2.token_logprobs_backward(g, x, t, saved, dentropy=g), lambda: oz2.token_logprobs_backward(g[:2], x, t, saved)):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: oz2.rms_norm(x.double(), w), lambda: oz2.rms_norm(x, w.half()), lambda: oz2.rms_norm(x, w, out_dtype=torch.int8),
              lambda: oz2.token_logprobs(x.long(), t), lambda: oz2.token_logprobs(x, t.int()),
              lambda: oz2.token_logprobs_backward(g.half(), x, t, saved)):
        with pytest.raises(TypeError):
            f()
