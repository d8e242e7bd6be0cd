"""The layer operators against their 64-bit definitions.

Tolerances are error bounds, element by element.  With u half an ulp of the
output type, a sum of k products in 32 bits is off by at most (k + 8) 2^-23
times the sum of the products' magnitudes (2^-23: the tensor cores' adder may
truncate), the activations by 2^-18 max(1, |z|) (the fast exponential and
quotient, with a margin), their slopes by 2^-17 (1 + |z|), and rounding adds
u times the result, or half the least subnormal.
"""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")
from tests._layers_ref import (TINY, UNIT, act, assert_within, keep_mask, norm_rope, slope)  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
SEED, OFFSET = 0x1234567890ABCDEF, 0x0FEDCBA987654321
ACC = 2.0**-23


@pytest.fixture(scope="module")
def oz2():
    import __graft_entry__ as g

    g.build()
    import emulated_fp64_gemm_gb300 as m

    assert torch.cuda.is_available()
    yield m
    assert m.last_error() == 0


def normal(*shape, dtype, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed + 17 * sum(shape))
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def strided(t, pad, shift):
    """t with rows `pad` elements longer apart and the first element `shift` elements into the storage."""
    rows, cols = t.shape
    store = torch.full((rows * (cols + pad) + shift + 8,), float("nan"), dtype=t.dtype, device=t.device)
    view = store[shift:].as_strided((rows, cols), (cols + pad, 1))
    view.copy_(t)
    return view


def factor(rows, cols, p):
    keep, scale = keep_mask(rows, cols, p, SEED, OFFSET)
    return keep.cuda(), scale


# ------------------------------------------------------------------ linear
def check_linear(oz2, x, w, bias, activation="none", residual=None, p=0.0, save=False, **kw):
    dtype, k = x.dtype, x.shape[1]
    u, tiny = UNIT[dtype], TINY[dtype]
    got = oz2.linear(x, w, bias, activation=activation, residual=residual, dropout=p, seed=SEED, offset=OFFSET,
                     save_preact=save, **kw)
    y, z_got = got if save else (got, None)
    z = x.double() @ w.double().t()
    mag = x.double().abs() @ w.double().abs().t()
    if bias is not None:
        z, mag = z + bias.double(), mag + bias.double().abs()
    z_err = (k + 8) * ACC * mag
    if save:
        assert_within(z_got, z, z_err + u * (z.abs() + z_err) + tiny, "preact")
    v = act(z, activation)
    err = 1.2 * z_err + (0 if activation in ("none", "relu") else 2.0**-18 * z.abs().clamp(min=1))
    if round(65536 * p):
        keep, scale = factor(*v.shape, p)
        v, err = torch.where(keep, v * scale, 0.0), torch.where(keep, err * scale + ACC * v.abs() * scale, 0.0)
    if residual is not None:
        v = v + residual.double()
    assert_within(y, v, err + (u + ACC) * (v.abs() + err) + tiny, "y")
    return y


SIZES = [(1, 1, 1), (1, 64, 128), (3, 8, 8), (2, 1000, 1000), (5, 33, 7), (16, 256, 512), (17, 264, 136), (33, 129, 257),
         (64, 2048, 192), (100, 72, 1024), (128, 512, 256), (129, 65, 100), (200, 4096, 8), (255, 320, 511), (256, 256, 256),
         (257, 1024, 264), (300, 8, 520), (515, 200, 1032), (1024, 1024, 1024)]


@pytest.mark.parametrize("m,k,n", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_linear_sizes(oz2, m, k, n, dtype):
    x, w, b = normal(m, k, dtype=dtype), normal(n, k, dtype=dtype, seed=1, scale=k**-0.5), normal(n, dtype=dtype, seed=2)
    r = normal(m, n, dtype=dtype, seed=3)
    check_linear(oz2, x, w, b)
    check_linear(oz2, x, w, b, "gelu_tanh", r, 0.25, save=True)


@pytest.mark.parametrize("m,k,n", [(3, 8200, 1000), (24, 4096, 20488), (120, 2056, 24640), (2000, 4104, 4360), (9000, 520, 2100)])
def test_linear_long(oz2, m, k, n):
    # more blocks of k than stages, more tiles than the device holds at once
    x, w, b = normal(m, k, dtype=BF16), normal(n, k, dtype=BF16, seed=1, scale=k**-0.5), normal(n, dtype=BF16, seed=2)
    check_linear(oz2, x, w, b, "silu", save=True)
    check_backward(oz2, normal(m, n, dtype=BF16, seed=3), x, w)


def test_linear_offsets_past_32_bits(oz2):
    # 2^31 elements of y and of the backward pass's dz, and more: rows at the far end against the same rows by themselves
    m, k, n = 70000, 64, 32768
    x, w, b = normal(m, k, dtype=BF16), normal(n, k, dtype=BF16, seed=1, scale=k**-0.5), normal(n, dtype=BF16, seed=2)
    y, z = oz2.linear(x, w, b, activation="silu", save_preact=True)
    for rows in (slice(0, 200), slice(65500, 65700), slice(m - 200, m)):
        want, want_z = oz2.linear(x[rows], w, b, activation="silu", save_preact=True)
        assert torch.equal(y[rows], want) and torch.equal(z[rows], want_z)
    dx, _, _ = oz2.linear_backward(y, x, w, preact=z, activation="silu", need_dw=False, need_dbias=False)
    rows = slice(m - 300, m)
    want, _, _ = oz2.linear_backward(y[rows], x[rows], w, preact=z[rows], activation="silu", need_dw=False, need_dbias=False)
    # the two calls may split their sums of 32768 terms differently: both are within the bound of the exact sums
    mag = y[rows].double().abs() @ w.double().abs() * 1.1
    assert_within(dx[rows], want.double(), 2 * (UNIT[BF16] * want.double().abs() + n * ACC * mag) + TINY[BF16], "dx")


@pytest.mark.parametrize("n", [2560, 2555])
def test_linear_split_tails(oz2, n):
    # 100 tiles of 256 x 256: the last ones are split along k and joined
    m, k = 2560, 4096
    x, w, b = normal(m, k, dtype=F16), normal(n, k, dtype=F16, seed=1, scale=k**-0.5), normal(n, dtype=F16, seed=2)
    r = normal(m, n, dtype=F16, seed=3)
    y = check_linear(oz2, x, w, b, "gelu", r, 0.1, save=True)
    assert torch.equal(y, oz2.linear(x, w, b, activation="gelu", residual=r, dropout=0.1, seed=SEED, offset=OFFSET))
    check_backward(oz2, normal(m, n, dtype=F16, seed=4), x, w)


@pytest.mark.parametrize("activation", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("m,n", [(4, 264), (300, 519)])
def test_linear_activations_and_options(oz2, activation, m, n):
    k = 136
    x, w = normal(m, k, dtype=BF16, scale=2.0), normal(n, k, dtype=BF16, seed=1, scale=2 * k**-0.5)
    b, r = normal(n, dtype=BF16, seed=2), normal(m, n, dtype=BF16, seed=3)
    check_linear(oz2, x, w, None, activation)
    check_linear(oz2, x, w, b, activation, save=True)
    check_linear(oz2, x, w, None, activation, r, 0.5)
    check_linear(oz2, x, w, b, activation, r, 1.0)


@pytest.mark.parametrize("m,k,n", [(7, 200, 300), (140, 320, 264), (700, 136, 520)])
@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (1, 0), (3, 5), (0, 1)])
def test_linear_strides(oz2, m, k, n, pad, shift):
    x, w = normal(m, k, dtype=F16), normal(n, k, dtype=F16, seed=1, scale=k**-0.5)
    r, b = normal(m, n, dtype=F16, seed=3), normal(n + shift, dtype=F16, seed=4)[shift:]
    out = strided(torch.zeros(m, n, dtype=F16, device="cuda"), pad, shift)
    y = check_linear(oz2, strided(x, pad, shift), strided(w, pad, shift), b, "relu", strided(r, pad, shift), 0.1, out=out)
    assert y is out
    assert torch.equal(y, oz2.linear(x, w, b, activation="relu", residual=r, dropout=0.1, seed=SEED, offset=OFFSET))
    # nothing is written between the rows
    between = out.as_strided((m - 1, pad), (n + pad, 1), out.storage_offset() + n) if pad else out[:0]
    assert bool(between.isnan().all())
    # column-major and broadcast operands are copied
    check_linear(oz2, x.t().contiguous().t(), w.t().contiguous().t(), b, residual=r[:1].expand(m, n))


@pytest.mark.parametrize("n", [264, 1027])
def test_linear_in_place_on_the_residual(oz2, n):
    for m in (5, 600, 5000):
        x, w, r = normal(m, 96, dtype=BF16), normal(n, 96, dtype=BF16, seed=1), normal(m, n, dtype=BF16, seed=2)
        want = oz2.linear(x, w, residual=r)
        assert torch.equal(oz2.linear(x, w, residual=r, out=r), want)


def test_linear_empty(oz2):
    w, b = normal(40, 24, dtype=BF16), normal(40, dtype=BF16)
    assert oz2.linear(normal(0, 24, dtype=BF16), w, b).shape == (0, 40)
    assert oz2.linear(normal(3, 24, dtype=BF16), w[:0], b[:0]).shape == (3, 0)
    # a sum over nothing is the bias
    y = oz2.linear(normal(3, 0, dtype=BF16), w[:, :0], b)
    assert torch.equal(y, b.expand(3, 40))


@pytest.mark.parametrize("m", [3, 200, 600])
def test_linear_special_values(oz2, m):
    k, n = 128, 264
    x, w = normal(m, k, dtype=BF16), normal(n, k, dtype=BF16, seed=1)
    r = normal(m, n, dtype=BF16, seed=2)
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    w[3, 9] = float("inf")
    w[:, 7] = 1.0
    x[:, 9] = x[:, 9].abs() + 0.5
    clean = [i for i in range(m) if i not in (1, 2)]
    y = oz2.linear(x, w, activation="relu", residual=r, dropout=0.5, seed=SEED, offset=OFFSET)
    keep, _ = factor(m, n, 0.5)
    assert bool(y[1][keep[1]].isnan().all())
    assert bool((y[2][keep[2]] == float("inf")).all())
    assert not bool(torch.isfinite(y[:, 3][keep[:, 3]]).any())
    # a dropped element is the residual, whatever the product was
    assert torch.equal(y[~keep], r[~keep])
    cols = [j for j in range(n) if j != 3]
    assert bool(torch.isfinite(y[clean][:, cols]).all())


def test_linear_large_values_saturate_like_the_formula(oz2):
    # activations of huge finite pre-activations: no NaN from inf * 0
    x = torch.tensor([[1e30], [-1e30], [3e4], [-3e4]], dtype=BF16, device="cuda")
    w = torch.ones(9, 1, dtype=BF16, device="cuda")
    for name in ("relu", "silu", "gelu", "gelu_tanh"):
        y = oz2.linear(x, w, activation=name)
        want = torch.where(x > 0, x, 0.0).expand(4, 9)
        assert torch.equal(y.abs(), want), name


def test_linear_streams_and_graph(oz2):
    x, w, r = normal(300, 512, dtype=BF16), normal(520, 512, dtype=BF16, seed=1), normal(300, 520, dtype=BF16, seed=2)
    want = oz2.linear(x, w, residual=r)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [oz2.linear(x, w, residual=r, stream=s) for _ in range(4)]
    with torch.cuda.stream(s):
        got.append(oz2.linear(x, w, residual=r))
    s.synchronize()
    assert all(torch.equal(g, want) for g in got)
    out = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        oz2.linear(x, w, residual=r, out=out)
        s.synchronize()
        with torch.cuda.graph(g, stream=s):
            oz2.linear(x, w, residual=r, out=out)
    out.zero_()
    x.copy_(-x)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, oz2.linear(x, w, residual=r))


# ------------------------------------------------------------------ linear_backward
def check_backward(oz2, dy, x, w, z=None, activation="none", p=0.0):
    dtype, u, tiny = dy.dtype, UNIT[dy.dtype], TINY[dy.dtype]
    (m, n), k = dy.shape, x.shape[1]
    got = oz2.linear_backward(dy, x, w, preact=z, activation=activation, dropout=p, seed=SEED, offset=OFFSET)
    dz, err = dy.double(), torch.zeros_like(dy, dtype=torch.float64)
    if activation != "none":
        sl = slope(z.double(), activation)
        err = dz.abs() * (0 if activation == "relu" else 2.0**-17 * (1 + z.double().abs()))
        dz = dz * sl
    if round(65536 * p):
        keep, scale = factor(m, n, p)
        dz, err = torch.where(keep, dz * scale, 0.0), torch.where(keep, err * scale + ACC * dz.abs() * scale, 0.0)
    if activation != "none" or round(65536 * p):
        rounded = err + u * (dz.abs() + err) + tiny  # dz as a 16-bit operand
    else:
        rounded = err
    for name, a, e, b, terms in (("dx", dz, rounded, w.double(), n), ("dw", dz.t(), rounded.t(), x.double(), m)):
        value, bound = a @ b, (e + (terms + 8) * ACC * (a.abs() + e)) @ b.abs()
        assert_within(got[0] if name == "dx" else got[1], value, bound + u * (value.abs() + bound) + tiny, name)
    value, bound = dz.sum(0), (err + (m + 8) * ACC * (dz.abs() + err)).sum(0)
    assert_within(got[2], value, bound + u * (value.abs() + bound) + tiny, "dbias")
    return got


@pytest.mark.parametrize("m,k,n", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_backward_sizes(oz2, m, k, n, dtype):
    x, w = normal(m, k, dtype=dtype), normal(n, k, dtype=dtype, seed=1, scale=k**-0.5)
    dy, z = normal(m, n, dtype=dtype, seed=2), normal(m, n, dtype=dtype, seed=3)
    check_backward(oz2, dy, x, w)
    check_backward(oz2, dy, x, w, z, "gelu_tanh", 0.25)


@pytest.mark.parametrize("activation", ["relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("p", [0.0, 0.3, 1.0])
def test_backward_activations(oz2, activation, p):
    m, k, n = 70, 40, 91
    check_backward(oz2, normal(m, n, dtype=BF16), normal(m, k, dtype=BF16, seed=1), normal(n, k, dtype=BF16, seed=2),
                   normal(m, n, dtype=BF16, seed=3, scale=2.0), activation, p)


@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (1, 0), (3, 5), (0, 1)])
def test_backward_strides(oz2, pad, shift):
    m, k, n = 270, 136, 264
    t = [strided(normal(*s, dtype=F16, seed=i), pad, shift) for i, s in enumerate(((m, n), (m, k), (n, k), (m, n)))]
    a = check_backward(oz2, *t[:3])
    b = oz2.linear_backward(*(v.contiguous() for v in t[:3]))
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    check_backward(oz2, *t, "silu")


# both products in one launch, the first or the second the one with the longer sums, k whole, in halves and in quarters
@pytest.mark.parametrize("m,k,n", [(65, 64, 65), (70, 200, 130), (130, 200, 70), (517, 130, 1531), (1024, 40, 1024), (3000, 8, 600),
                                   (600, 8, 3000), (129, 1000, 257)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_backward_products_side_by_side(oz2, m, k, n, dtype):
    x, w = normal(m, k, dtype=dtype), normal(n, k, dtype=dtype, seed=1, scale=k**-0.5)
    dy, z = normal(m, n, dtype=dtype, seed=2), normal(m, n, dtype=dtype, seed=3)
    a = check_backward(oz2, dy, x, w)
    b = oz2.linear_backward(dy, x, w)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    check_backward(oz2, dy, x, w, z, "silu", 0.25)


def test_backward_parts_and_empty(oz2):
    m, k, n = 33, 72, 50
    dy, x, w = normal(m, n, dtype=BF16), normal(m, k, dtype=BF16, seed=1), normal(n, k, dtype=BF16, seed=2)
    full = oz2.linear_backward(dy, x, w)
    for i, name in enumerate(("need_dx", "need_dw", "need_dbias")):
        flags = {f: f == name for f in ("need_dx", "need_dw", "need_dbias")}
        part = oz2.linear_backward(dy, x, w, **flags)
        assert torch.equal(part[i], full[i]) and all(part[j] is None for j in range(3) if j != i)
    # no rows: gradients of sums over nothing
    dx, dw, db = oz2.linear_backward(dy[:0], x[:0], w)
    assert dx.shape == (0, k) and not dw.any() and not db.any()
    dx, dw, db = oz2.linear_backward(dy[:, :0], x, w[:0])
    assert not dx.any() and dw.shape == (0, k) and db.shape == (0,)
    dx, dw, db = oz2.linear_backward(dy, x[:, :0], w[:, :0])
    assert dx.shape == (m, 0) and torch.equal(db, full[2])


def test_backward_dropped_elements_give_nothing(oz2):
    # NaN and inf at dropped places do not reach any gradient
    m, k, n = 40, 64, 48
    dy, x, w, z = (normal(*s, dtype=BF16, seed=i) for i, s in enumerate(((m, n), (m, k), (n, k), (m, n))))
    keep, _ = factor(m, n, 0.5)
    want = oz2.linear_backward(dy, x, w, preact=z, activation="silu", dropout=0.5, seed=SEED, offset=OFFSET)
    dy[~keep], z[~keep] = float("nan"), float("inf")
    got = oz2.linear_backward(dy, x, w, preact=z, activation="silu", dropout=0.5, seed=SEED, offset=OFFSET)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("activation", ["silu", "gelu", "gelu_tanh"])
def test_backward_against_differences(oz2, activation):
    """Gradients along random directions against central differences of the 64-bit definition."""
    m, k, n = 24, 32, 40
    x, w, b, dy = (normal(*s, dtype=F16, seed=i) for i, s in enumerate(((m, k), (n, k), (n,), (m, n))))
    w = (w * 0.2).to(F16)
    keep, scale = factor(m, n, 0.2)

    def loss(x, w, b):
        return float((torch.where(keep, act(x @ w.t() + b, activation) * scale, 0.0) * dy.double()).sum())

    _, z = oz2.linear(x, w, b, activation=activation, dropout=0.2, seed=SEED, offset=OFFSET, save_preact=True)
    grads = oz2.linear_backward(dy, x, w, preact=z, activation=activation, dropout=0.2, seed=SEED, offset=OFFSET)
    at = [t.double() for t in (x, w, b)]
    for i, g in enumerate(grads):
        d = normal(*at[i].shape, dtype=F32, seed=9 + i).double()
        h = 1e-4
        up, down = ([t + s * h * d if j == i else t for j, t in enumerate(at)] for s in (1, -1))
        diff = (loss(*up) - loss(*down)) / (2 * h)
        # every element of the gradient carries a relative rounding of 2^-11 from its output, from dz and from z (whose
        # rounding shifts the slope, |act''| <= 1.2, by up to 2^-10): well inside 2^-8 of the sum of magnitudes
        assert abs(float((g.double() * d).sum()) - diff) <= 2.0**-8 * float((g.double().abs() * d.abs()).sum()) + 1e-6


# ------------------------------------------------------------------ dropout
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7), (3, 8), (5, 9), (64, 1000), (257, 264), (1000, 33)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
def test_dropout(oz2, rows, cols, dtype, p):
    x, r = normal(rows, cols, dtype=dtype), normal(rows, cols, dtype=dtype, seed=1)
    keep, scale = factor(rows, cols, p)
    v = torch.where(keep, x.double() * scale, 0.0)
    u = UNIT[dtype]
    # the scale, the product and (with a residual) the sum are rounded to 32 bits each, the result once to its type
    assert_within(oz2.dropout(x, p, seed=SEED, offset=OFFSET), v, (u + 2.0**-22) * v.abs() + TINY[dtype])
    want = v + r.double()
    assert_within(oz2.dropout(x, p, seed=SEED, offset=OFFSET, residual=r), want,
                  (u + 2.0**-23) * want.abs() + 2.0**-22 * v.abs() + TINY[dtype])
    dx = oz2.dropout_backward(x, p, seed=SEED, offset=OFFSET)
    assert torch.equal(dx, oz2.dropout(x, p, seed=SEED, offset=OFFSET))
    assert bool((dx[~keep] == 0).all())


def test_dropout_strides_in_place_and_special_values(oz2):
    x, r = normal(100, 264, dtype=BF16), normal(100, 264, dtype=BF16, seed=1)
    want = oz2.dropout(x, 0.3, seed=SEED, offset=OFFSET, residual=r)
    for pad, shift in ((8, 0), (8, 8), (1, 0), (3, 5)):
        out = strided(torch.zeros_like(x), pad, shift)
        assert torch.equal(oz2.dropout(strided(x, pad, shift), 0.3, seed=SEED, offset=OFFSET, residual=strided(r, pad, shift), out=out), want)
    y = x.clone()
    assert oz2.dropout(y, 0.3, seed=SEED, offset=OFFSET, residual=r, out=y) is y and torch.equal(y, want)
    assert torch.equal(oz2.dropout(x.t().contiguous().t(), 0.3, seed=SEED, offset=OFFSET, residual=r), want)
    assert torch.equal(oz2.dropout(x, 0.3, seed=SEED - 2**64, offset=OFFSET, residual=r), want)
    assert not torch.equal(oz2.dropout(x, 0.3, seed=SEED, offset=OFFSET + 1, residual=r), want)
    keep, _ = factor(100, 264, 0.3)
    x[~keep] = float("nan")
    assert torch.equal(oz2.dropout(x, 0.3, seed=SEED, offset=OFFSET, residual=r), want)
    assert oz2.dropout(x[:0], 0.3, seed=1).shape == (0, 264) and oz2.dropout(x[:, :0], 0.3, seed=1).shape == (100, 0)


@pytest.mark.parametrize("rows,cols,ld", [(37, 64, 65), (5, 256, 259), (9, 257, 257), (21, 261, 263), (33, 1001, 1001), (3, 2050, 2051),
                                          (600, 5001, 5001), (2, 70001, 70003), (1, 1000, 1000)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_dropout_rows_off_boundaries(oz2, rows, cols, ld, dtype):
    # matrices whose rows are alike off their boundaries, from each start, against the same call with rows that differ
    x, r = normal(rows, cols, dtype=dtype), normal(rows, cols, dtype=dtype, seed=1)
    want = oz2.dropout(x, 0.3, seed=SEED, offset=OFFSET, residual=r)
    keep, scale = factor(rows, cols, 0.3)
    exact = torch.where(keep, x.double() * scale, 0.0) + r.double()
    assert_within(want, exact, (UNIT[dtype] + 2.0**-23) * exact.abs() + 2.0**-22 * (exact - r.double()).abs() + TINY[dtype])
    plain = oz2.dropout(x, 0.3, seed=SEED, offset=OFFSET)
    copied = oz2.dropout(x, 0.0, seed=SEED, residual=r)

    def at(start, values=None):
        buffer = torch.full((rows * ld + 16,), -7.0, dtype=dtype, device="cuda")
        view = buffer.as_strided((rows, cols), (ld, 1), start)
        if values is not None:
            view.copy_(values)
        return buffer, view

    for start in range(8):
        for y_start in (start, start + 3):
            (buffer, y), xs, rs = at(y_start), at(start, x)[1], at(start, r)[1]
            assert torch.equal(oz2.dropout(xs, 0.3, seed=SEED, offset=OFFSET, residual=rs, out=y), want)
            y.fill_(-7.0)
            assert bool((buffer == -7.0).all()), "nothing beside the rows is written"
            assert torch.equal(oz2.dropout(xs, 0.3, seed=SEED, offset=OFFSET, out=y), plain)
        assert torch.equal(oz2.dropout(xs, 0.0, seed=SEED, residual=rs, out=at(start)[1]), copied)
        assert torch.equal(oz2.dropout(xs, 0.3, seed=SEED, offset=OFFSET, residual=rs, out=xs), want)


def test_dropout_rate_and_row_numbers(oz2):
    # kept shares by row, by column within a group and in all, within six standard deviations
    x = torch.ones(4096, 2048, dtype=BF16, device="cuda")
    kept = (oz2.dropout(x, 0.25, seed=5) != 0).double()
    for mean, count in ((kept.mean(), kept.numel()), (kept.mean(1), 2048), (kept.reshape(-1, 8).mean(0), kept.numel() / 8)):
        assert float((mean - 0.75).abs().max()) <= 6 * math.sqrt(0.25 * 0.75 / count)
    # rows and layers do not repeat one another's mask
    assert not torch.equal(kept[0], kept[1])
    assert not torch.equal(kept, (oz2.dropout(x, 0.25, seed=6) != 0).double())


def test_dropout_offsets_past_32_bits(oz2):
    # 2^31 elements and more: element offsets need 64 bits (bytes past 2^32)
    rows, cols = 70000, 32768
    x = torch.ones(rows, cols, dtype=BF16, device="cuda")
    y = oz2.dropout(x, 0.5, seed=SEED, offset=OFFSET, out=x)
    keep, _ = keep_mask(1, cols, 0.5, SEED, OFFSET)
    assert torch.equal(y[0].cpu() != 0, keep[0])
    tail = oz2.dropout(torch.ones(rows, 8, dtype=BF16, device="cuda"), 0.5, seed=SEED, offset=OFFSET)
    assert torch.equal(y[:, :8], tail)
    assert abs(float((y[-1000:] != 0).float().mean()) - 0.5) < 0.001


# ------------------------------------------------------------------ qk_norm_rope
def tables(rows, rot):
    a = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * torch.exp(
        torch.arange(rot // 2, device="cuda", dtype=torch.float64) * (-2.0 * math.log(10000.0) / max(rot, 1)))
    return a.cos().float(), a.sin().float()


def qk_inputs(t, hq, hkv, d, rot, dtype, rows=512):
    qkv = normal(t, hq + 2 * hkv, d, dtype=dtype)
    q, k = qkv[:, :hq], qkv[:, hq:hq + hkv]
    wq, wk = 1 + 0.1 * normal(d, dtype=dtype, seed=1), 1 + 0.1 * normal(d, dtype=dtype, seed=2)
    cos, sin = tables(rows, rot)
    pos = torch.randint(0, rows, (t,), generator=torch.Generator(device="cuda").manual_seed(t), device="cuda")
    return q, k, wq, wk, cos, sin, pos


QK = [(1, 1, 1, 128, 128), (3, 4, 1, 64, 64), (24, 32, 8, 128, 128), (7, 3, 2, 96, 64), (5, 2, 2, 80, 80), (9, 1, 1, 2, 2),
      (11, 3, 1, 1, 0), (33, 5, 5, 37, 16), (6, 8, 2, 256, 64), (130, 2, 1, 512, 512), (2, 1, 1, 511, 510), (300, 16, 4, 72, 24),
      (40, 12, 0, 128, 64), (40, 0, 3, 64, 32), (1000, 7, 1, 104, 0)]


@pytest.mark.parametrize("t,hq,hkv,d,rot", QK)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_qk_norm_rope_and_gradients(oz2, t, hq, hkv, d, rot, interleaved, dtype):
    q, k, wq, wk, cos, sin, pos = qk_inputs(t, hq, hkv, d, rot, dtype)
    u, eps = UNIT[dtype], 1e-5
    got = oz2.qk_norm_rope(q, k, wq, wk, cos, sin, pos, eps=eps, interleaved=interleaved)
    leaves = [v.double().requires_grad_(True) for v in (q, k, wq, wk)]
    c, s = cos[pos], sin[pos]
    want = [norm_rope(leaves[i], leaves[2 + i], c, s, eps, interleaved) for i in range(2)]
    dq, dk = normal(t, hq, d, dtype=dtype, seed=7), normal(t, hkv, d, dtype=dtype, seed=8)
    grads = torch.autograd.grad(want, leaves, (dq.double(), dk.double()))
    back = oz2.qk_norm_rope_backward(dq, dk, q, k, wq, wk, cos, sin, pos, eps=eps, interleaved=interleaved)
    # forward: r is off by (d + 8) 2^-24 relatively at most, the products and the rotation by a few units of 2^-24 of the
    # pair's size, which the norm bounds: |u| <= sqrt(d) max|w|.  Errors average far lower; this is the worst case.
    for i, (x, w) in enumerate(((q, wq), (k, wk))):
        if x.numel() == 0:
            assert got[i].numel() == 0
            continue
        size = norm_rope(x.double(), w.double(), c, s, eps, interleaved).abs()
        pair = (x.double() * w.double()).abs() / torch.sqrt((x.double()**2).mean(-1, keepdim=True) + eps)
        pair = pair.amax(-1, keepdim=True)
        e = (d + 24) * 2.0**-24
        assert_within(got[i], want[i].detach(), u * size + 2 * e * pair + TINY[dtype], "forward")
        # gradients: g and the mean of g w x carry the same kinds of error, times r and the largest g w
        gw = (dq if i == 0 else dk).double().abs().amax(-1, keepdim=True) * w.double().abs().max() * 2
        r = 1 / torch.sqrt((x.double()**2).mean(-1, keepdim=True) + eps)
        xr = (x.double().abs() * r)
        bound = 4 * e * r * gw * (1 + xr * xr.amax(-1, keepdim=True))
        assert_within(back[i], grads[i], u * grads[i].abs() * (1 + e) + bound + TINY[dtype], "dx")
        terms = t * x.shape[1]
        mag = ((dq if i == 0 else dk).double().abs().amax(-1, keepdim=True) * 2 * xr).sum((0, 1))
        assert_within(back[2 + i], grads[2 + i], u * grads[2 + i].abs() * (1 + e) + (2 * e + (terms + 8) * 2.0**-24) * mag + TINY[dtype],
                      "dweight")


def test_qk_in_place_strides_and_positions(oz2):
    q, k, wq, wk, cos, sin, pos = qk_inputs(50, 6, 2, 64, 32, BF16)
    want = oz2.qk_norm_rope(q, k, wq, wk, cos, sin, pos)
    # heads before tokens, features apart (copied), a view that starts off a 16-byte boundary
    for f in (lambda v: v.transpose(0, 1).contiguous().transpose(0, 1), lambda v: v.transpose(1, 2).contiguous().transpose(1, 2),
              lambda v: torch.nn.functional.pad(v, (3, 2))[..., 3:-2]):
        got = oz2.qk_norm_rope(f(q), f(k), wq, wk, cos, sin, pos)
        assert all(torch.allclose(a.float(), b.float(), rtol=2**-7, atol=1e-6) for a, b in zip(got, want))
    qkv = torch.cat((q, k), 1)
    oz2.qk_norm_rope(qkv[:, :6], qkv[:, 6:], wq, wk, cos, sin, pos, out=(qkv[:, :6], qkv[:, 6:]))
    assert torch.equal(qkv[:, :6], want[0]) and torch.equal(qkv[:, 6:], want[1])
    # positions outside the tables: NaN in their tokens, the others untouched
    bad = pos.clone()
    bad[3], bad[9], bad[11] = -1, 512, 2**40
    got = oz2.qk_norm_rope(q, k, wq, wk, cos, sin, bad)
    ok = [i for i in range(50) if i not in (3, 9, 11)]
    for a, b in zip(got, want):
        assert bool(a[[3, 9, 11]].isnan().all()) and torch.equal(a[ok], b[ok])
    # an empty batch, and rows of zeros (the norm's eps)
    e = oz2.qk_norm_rope(q[:0], k[:0], wq, wk, cos, sin, pos[:0])
    assert e[0].shape == (0, 6, 64)
    g = oz2.qk_norm_rope_backward(e[0], e[1], q[:0], k[:0], wq, wk, cos, sin, pos[:0])
    assert not g[2].any() and not g[3].any()
    z = oz2.qk_norm_rope(torch.zeros_like(q), torch.zeros_like(k), wq, wk, cos, sin, pos)
    assert not z[0].any() and not z[1].any()


def test_qk_backward_is_repeatable_and_in_place(oz2):
    q, k, wq, wk, cos, sin, pos = qk_inputs(3000, 8, 2, 128, 128, BF16)
    dq, dk = normal(3000, 8, 128, dtype=BF16, seed=4), normal(3000, 2, 128, dtype=BF16, seed=5)
    a = oz2.qk_norm_rope_backward(dq, dk, q, k, wq, wk, cos, sin, pos)
    b = oz2.qk_norm_rope_backward(dq, dk, q, k, wq, wk, cos, sin, pos)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    joint = torch.zeros(3000, 12, 128, dtype=BF16, device="cuda")
    c = oz2.qk_norm_rope_backward(dq, dk, q, k, wq, wk, cos, sin, pos, out=(joint[:, :8], joint[:, 8:10]))
    assert torch.equal(joint[:, :8], a[0]) and torch.equal(joint[:, 8:10], a[1]) and not joint[:, 10:].any()
    assert torch.equal(c[2], a[2])


def test_qk_backward_against_differences(oz2):
    q, k, wq, wk, cos, sin, pos = qk_inputs(12, 3, 2, 48, 32, F32)
    dq, dk = normal(12, 3, 48, dtype=F32, seed=4), normal(12, 2, 48, dtype=F32, seed=5)
    grads = oz2.qk_norm_rope_backward(dq, dk, q, k, wq, wk, cos, sin, pos, interleaved=True)
    at = [v.double() for v in (q, k, wq, wk)]

    def loss(q, k, wq, wk):
        c, s = cos[pos], sin[pos]
        return float((norm_rope(q, wq, c, s, 1e-6, True) * dq.double()).sum() + (norm_rope(k, wk, c, s, 1e-6, True) * dk.double()).sum())

    for i, g in enumerate(grads):
        d = normal(*at[i].shape, dtype=F32, seed=20 + i).double()
        up, down = ([v + s * 1e-5 * d if j == i else v for j, v in enumerate(at)] for s in (1, -1))
        diff = (loss(*up) - loss(*down)) / 2e-5
        # 32-bit gradients and a central difference with h = 1e-5: relative 1e-5 of the sum of magnitudes
        assert abs(float((g.double() * d).sum()) - diff) <= 1e-5 * float((g.double().abs() * d.abs()).sum())


@pytest.mark.parametrize("t,hq,hkv,d,rot", [(700, 8, 8, 128, 128), (5000, 3, 1, 64, 64)])
def test_qk_equal_positions_and_long_runs(oz2, t, hq, hkv, d, rot):
    # all tokens at one position, more steps per warp than are in flight; against each token by itself
    q, k, wq, wk, cos, sin, _ = qk_inputs(t, hq, hkv, d, rot, BF16)
    pos = torch.full((t,), 77, device="cuda")
    got = oz2.qk_norm_rope(q, k, wq, wk, cos, sin, pos)
    for i in (0, 1, t // 2, t - 1):
        one = oz2.qk_norm_rope(q[i:i + 1], k[i:i + 1], wq, wk, cos, sin, pos[:1])
        assert torch.equal(got[0][i], one[0][0]) and torch.equal(got[1][i], one[1][0])


# ------------------------------------------------------------------ together
def test_block_example(oz2):
    """The example's block: its gradients against 64-bit autograd of the same block, its training and its single tokens."""
    import importlib.util
    import os

    from tests._util import ROOT

    spec = importlib.util.spec_from_file_location("transformer_block", os.path.join(ROOT, "examples", "transformer_block.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    block = ex.Block(dim=256, heads=4, kv_heads=2, hidden=768)
    t, p = 64, 0.1
    x = normal(t, 256, dtype=BF16)
    pos = torch.arange(t, device="cuda")
    dy = normal(t, 256, dtype=BF16, seed=1)
    y = block(x, pos, p, seed=SEED, step=3)
    grads = torch.autograd.grad(y, list(block.w.values()), dy)

    w = {n: v.detach().double().requires_grad_(True) for n, v in block.w.items()}
    h, kv, d = block.heads, block.kv_heads, block.head_dim

    def drop(v, i):
        keep, scale = keep_mask(*v.shape, p, SEED, 4 * 3 + i)
        return torch.where(keep.cuda(), v * scale, 0.0)

    x0 = drop(x.double(), 0)
    qkv = (x0 @ w["qkv"].t() + w["qkv_b"]).view(t, h + 2 * kv, d)
    q = norm_rope(qkv[:, :h], w["wq"], block.cos[pos], block.sin[pos], 1e-6, False)
    k = norm_rope(qkv[:, h:h + kv], w["wk"], block.cos[pos], block.sin[pos], 1e-6, False).repeat_interleave(h // kv, 1)
    v = qkv[:, h + kv:].repeat_interleave(h // kv, 1)
    s = torch.einsum("thd,shd->hts", q, k) * d**-0.5 + torch.full((t, t), float("-inf"), device="cuda").triu(1)
    o = torch.einsum("hts,shd->thd", s.softmax(-1), v).flatten(1)
    x1 = x0 + drop(o @ w["out"].t() + w["out_b"], 1)
    want = x1 + drop(act(x1 @ w["up"].t() + w["up_b"], "gelu_tanh") @ w["down"].t() + w["down_b"], 2)
    exact = torch.autograd.grad(want, list(w.values()), dy.double())
    # a chain of about ten bfloat16 roundings of 2^-9 each: 2 % of the norm is four times their sum
    for name, got, ref in (("y", y, want), *zip(w, grads, exact)):
        got, ref = got.detach().double(), ref.detach()
        assert float((got - ref).norm()) <= 0.02 * float(ref.norm()), name
    losses = ex.train(block, tokens=64, steps=6)
    assert losses[-1] < losses[0]
    with torch.no_grad():
        whole = block(x, pos)
    single = ex.decode(block, x)
    assert float((whole.double() - single.double()).norm()) <= 0.02 * float(whole.double().norm())


# ------------------------------------------------------------------ refusals
def test_refusals(oz2):
    x, w, b, r = normal(4, 16, dtype=BF16), normal(8, 16, dtype=BF16), normal(8, dtype=BF16), normal(4, 8, dtype=BF16)
    before = oz2.launch_count()
    bad = [
        (TypeError, lambda: oz2.linear(x.float(), w.float())),
        (TypeError, lambda: oz2.linear(x, w.half())),
        (TypeError, lambda: oz2.linear(x, w, b.float())),
        (ValueError, lambda: oz2.linear(x, w[:, :8])),
        (ValueError, lambda: oz2.linear(x[0], w)),
        (ValueError, lambda: oz2.linear(x.cpu(), w)),
        (ValueError, lambda: oz2.linear(x, w.cpu())),
        (ValueError, lambda: oz2.linear(x, w, b[:4])),
        (ValueError, lambda: oz2.linear(x, w, residual=r[:, :4])),
        (ValueError, lambda: oz2.linear(x, w, activation="tanh")),
        (ValueError, lambda: oz2.linear(x, w, dropout=1.5)),
        (ValueError, lambda: oz2.linear(x, w, dropout=float("nan"))),
        (ValueError, lambda: oz2.linear(x, w, out=torch.empty(8, 4, dtype=BF16, device="cuda").t())),
        (ValueError, lambda: oz2.linear_backward(r, x, w, activation="silu")),
        (ValueError, lambda: oz2.linear_backward(r, x[:3], w)),
        (ValueError, lambda: oz2.linear_backward(r, x, w[:4])),
        (TypeError, lambda: oz2.linear_backward(r, x, w, preact=r.float(), activation="silu")),
        (ValueError, lambda: oz2.dropout(x, -0.1, seed=1)),
        (TypeError, lambda: oz2.dropout(x.double(), 0.1, seed=1)),
        (ValueError, lambda: oz2.dropout(x, 0.1, seed=1, residual=r)),
    ]
    q, k, wq, wk, cos, sin, pos = qk_inputs(4, 2, 1, 16, 16, BF16)
    bad += [
        (TypeError, lambda: oz2.qk_norm_rope(q, k, wq.float(), wk, cos, sin, pos)),
        (TypeError, lambda: oz2.qk_norm_rope(q, k, wq, wk, cos.half(), sin, pos)),
        (TypeError, lambda: oz2.qk_norm_rope(q, k, wq, wk, cos, sin, pos.int())),
        (ValueError, lambda: oz2.qk_norm_rope(q, k[:3], wq, wk, cos, sin, pos)),
        (ValueError, lambda: oz2.qk_norm_rope(q, k, wq, wk, cos, sin[:, :4], pos)),
        (ValueError, lambda: oz2.qk_norm_rope(q, k, wq, wk, *tables(8, 32), pos)),
        (ValueError, lambda: oz2.qk_norm_rope(q, k, wq, wk, cos, sin, pos[:2])),
        (ValueError, lambda: oz2.qk_norm_rope(q, k, wq, wk, cos, sin, pos, out=(torch.empty_like(q[:2]), None))),
        (oz2.Ozaki2Error, lambda: oz2.qk_norm_rope(q, k, wq, wk, cos, sin, pos, eps=-1.0)),
        (ValueError, lambda: oz2.qk_norm_rope_backward(q[:2], k, q, k, wq, wk, cos, sin, pos)),
    ]
    for kind, f in bad:
        with pytest.raises(kind):
            f()
    assert oz2.launch_count() == before
