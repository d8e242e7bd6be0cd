"""The layer operators where they leave the ordinary path: waits that run out, the ends of
the types' ranges, activations' tails, positions out of range, and what autograd is told."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")
from tests._layers_ref import TINY, UNIT, assert_within, keep_mask, slope  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
SEED, OFFSET = 0x1234567890ABCDEF, 0x0FEDCBA987654321


@pytest.fixture(scope="module")
def oz2():
    import __graft_entry__ as g

    g.build()
    import emulated_fp64_gemm_gb300 as m

    assert torch.cuda.is_available()
    yield m
    assert m.last_error() == 0


def normal(*shape, dtype=BF16, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed + 13 * sum(shape))
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


# ------------------------------------------------------------------ waits that run out
@pytest.mark.parametrize("limit_us", [50, 5000])
def test_product_kernels_wind_down_when_their_operands_never_come(oz2, limit_us):
    x, w = normal(700, 512), normal(520, 512, seed=1)
    few = normal(9, 512, seed=2)
    want, want_few = oz2.linear(x, w), oz2.linear(few, w)
    before = oz2.launch_count()
    assert oz2.selftest_wait_timeout(limit_us) == 5
    assert oz2.launch_count() - before == 3  # a plain wait, and one product of each form
    # their tensor memory is free again and nothing of them arrives later
    assert oz2.last_error() == 0
    for _ in range(3):
        assert torch.equal(oz2.linear(x, w), want) and torch.equal(oz2.linear(few, w), want_few)


# ------------------------------------------------------------------ the ends of the types' ranges
def check_backward(oz2, dy, x, w, z, activation, p, seed, offset):
    """dx and dw against the 64-bit definition.

    With u half an ulp of the type: dz is rounded to it once, without the
    dropout's scale (relative u, and at most half the least subnormal times that
    scale and the activations' common factor, together below 4 for these p); its
    slope is off by 2^-17 (1 + |z|); sums of t products in 32 bits by (t + 8)
    2^-23 of their magnitudes; the outputs are rounded once."""
    dtype, u, tiny = dy.dtype, UNIT[dy.dtype], TINY[dy.dtype]
    (m, n), k = dy.shape, x.shape[1]
    dx, dw, db = oz2.linear_backward(dy, x, w, preact=z, activation=activation, dropout=p, seed=seed, offset=offset)
    dz, err = dy.double(), torch.zeros(m, n, dtype=torch.float64, device="cuda")
    if z is not None:
        if activation != "relu":
            err = dz.abs() * 2.0**-17 * (1 + z.double().abs())
        dz = dz * slope(z.double(), activation)
    if p:
        keep, scale = keep_mask(m, n, p, seed, offset)
        dz, err = (torch.where(keep.cuda(), v * scale, 0.0) for v in (dz, err))
    err = err + (u + 2.0**-22) * (dz.abs() + err) + 4 * tiny
    for name, got, a, e, b, terms in (("dx", dx, dz, err, w.double(), n), ("dw", dw, dz.t(), err.t(), x.double(), m)):
        value, bound = a @ b, (e + (terms + 8) * 2.0**-23 * (a.abs() + e)) @ b.abs()
        assert_within(got, value, bound + u * (value.abs() + bound) + tiny, name)
    return dx, dw, db


@pytest.mark.parametrize("m,k,n", [(40, 72, 96), (150, 136, 264), (700, 520, 1032)])
@pytest.mark.parametrize("activation,p,top", [("none", 0.5, 6e4), ("relu", 0.75, 6e4), ("silu", 0.5, 6.5e4), ("gelu", 0.0, 6.55e4),
                                              ("gelu_tanh", 0.1, 6.55e4)])
def test_backward_of_gradients_near_the_largest_float16(oz2, m, k, n, activation, p, top):
    # dz itself passes the largest float16 (by the dropout's scale, by the activation's slope up to 1.13), the gradients do not
    dy = (torch.rand(m, n, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") * 0.05 + 0.95) * top
    dy = (dy * torch.where(torch.arange(n, device="cuda") % 2 == 0, 1.0, -1.0)).to(F16)
    z = (1.0 + normal(m, n, dtype=F32, seed=2).abs()).to(F16)  # slopes around their largest
    x, w = normal(m, k, dtype=F16, seed=3, scale=2.0**-14), normal(n, k, dtype=F16, seed=4, scale=2.0**-10)
    x[0, 0], w[0, 0] = 0.0, 0.0
    dx, dw, db = check_backward(oz2, dy, x, w, None if activation == "none" else z, activation, p, SEED, OFFSET)
    assert bool(torch.isfinite(dx).all()) and bool(torch.isfinite(dw).all())
    # (dbias passes the range in its own right: its sums are the definition's)


@pytest.mark.parametrize("p", [0.0, 0.5])
def test_backward_of_gradients_near_the_least_float16(oz2, p):
    # dz of subnormal size: off by half the least subnormal where it is rounded, no more
    m, k, n = 130, 64, 200
    dy, z = normal(m, n, dtype=F16, scale=2.0**-17), normal(m, n, dtype=F16, seed=2)
    x, w = normal(m, k, dtype=F16, seed=3, scale=64.0), normal(n, k, dtype=F16, seed=4, scale=64.0)
    check_backward(oz2, dy, x, w, z, "silu", p, SEED, OFFSET)


# ------------------------------------------------------------------ activations over every finite value
C2, A3 = 2 * math.sqrt(2 / math.pi), 0.044715


def every_value(dtype):
    bits = torch.arange(-32768, 32768, device="cuda").to(torch.int16)
    v = bits.view(dtype)
    return v[torch.isfinite(v)].reshape(-1, 1)


def exact_activation(z, name):
    """act(z), act'(z), the size of the slope's terms, and the size of the exponent that their tails are made by.

    All are free of cancellation in the tails.  For large z the factor is exactly
    1 in 32 bits, so that the sizes stop growing there."""
    if name == "relu":
        return z.clamp(min=0), (z > 0).double(), torch.ones_like(z), torch.zeros_like(z)
    if name == "gelu":
        cdf = 0.5 * torch.special.erfc(-z * math.sqrt(0.5))
        bell = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        return z * cdf, cdf + z * bell, cdf + z.abs() * bell, z.clamp(max=6)**2
    if name == "silu":
        s, near = torch.sigmoid(z), z.clamp(max=20)
        return z * s, s + z * s * torch.sigmoid(-z), s * (1 + near.abs()), near.abs()
    near = z.clamp(max=5.1)
    argument, limited = C2 * (z + A3 * z**3), C2 * (near + A3 * near**3).abs()
    s, g, g_near = torch.sigmoid(argument), C2 * (1 + 3 * A3 * z * z), C2 * (1 + 3 * A3 * near * near)
    # far out g times sigmoid(-argument) would be infinity times zero
    bend = torch.where(argument.abs() > 700, 0.0, z * s * torch.sigmoid(-argument) * g)
    return z * s, s + bend, torch.where(argument < -700, 0.0, s * (1 + near.abs() * g_near)), limited


@pytest.mark.parametrize("activation", ["relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_activations_relatively_over_every_finite_value(oz2, activation, dtype):
    """A product with 1 is exact, so what is left is the activation and one rounding.

    Its factor is off by at most 2^-18 relatively (a fit of 2^-20.3, a dozen
    roundings of 2^-24, the approximate exponential and reciprocal of 2^-22),
    and by the exponent's own roundings: at most eight of 2^-24 times its size.
    Factors below the least normal number, 2^-126, come out as zero."""
    u, tiny = UNIT[dtype], TINY[dtype]
    x = every_value(dtype)
    z = x.double()
    want, rise, terms, exponent = exact_activation(z, activation)
    rel = 0.0 if activation == "relu" else 2.0**-18 + exponent * 2.0**-21
    one = torch.ones(1, 1, dtype=dtype, device="cuda")
    y = oz2.linear(x, one, activation=activation)
    assert_within(y, want, (rel + u * (1 + rel)) * want.abs() + tiny + z.abs() * 2.0**-126, "value")
    # the slopes through dz and the product with 1: two roundings, the first of dz or of 7/8 of it
    dx, _, _ = oz2.linear_backward(torch.ones_like(x), x, one, preact=x, activation=activation, need_dw=False, need_dbias=False)
    err = rel * terms + (1 + z.abs() * C2 * (1 + 3 * A3 * z * z)).clamp(max=2.0**30) * 2.0**-126
    assert_within(dx, rise, err + 2.1 * u * (rise.abs() + err) + 2.2 * tiny, "slope")


def test_gelu_tail_relatively(oz2):
    # 32-bit sums between the 16-bit values: z = x w, -12 to 12, against the distribution function's own tail
    x = torch.linspace(-12, 12, 4001, device="cuda").to(BF16).reshape(-1, 1)
    w = (1 + torch.arange(64, device="cuda") / 256.0).clamp(max=1.25).to(BF16).reshape(-1, 1)
    z = x.double() @ w.double().t()
    want, _, _, exponent = exact_activation(z, "gelu")
    rel = 2.0**-18 + (exponent + 1) * 2.0**-21
    # (the product is exact: both have eight significant bits)
    assert_within(oz2.linear(x, w, activation="gelu"), want, (rel + UNIT[BF16] * (1 + rel)) * want.abs() + TINY[BF16] + z.abs() * 2.0**-126)


# ------------------------------------------------------------------ residuals of long products
@pytest.mark.parametrize("m,n", [(4133, 4104), (4352, 4360), (700, 1032)])
@pytest.mark.parametrize("in_place", [False, True])
def test_residual_of_long_products_with_ragged_ends(oz2, m, n, in_place):
    # more than 256 k blocks per pair of SMs (the form with fewer epilogue warps), and fewer; blocks past the rows' and columns' ends
    k = 4352
    x, w, r = normal(m, k), normal(n, k, seed=1, scale=k**-0.5), normal(m, n, seed=2)
    z = x.double() @ w.double().t()
    want = z.clamp(min=0) + r.double()
    err = 1.2 * (k + 8) * 2.0**-23 * (x.double().abs() @ w.double().abs().t())
    y = oz2.linear(x, w, activation="relu", residual=r, out=r if in_place else None)
    assert_within(y, want, err + (UNIT[BF16] + 2.0**-23) * (want.abs() + err) + TINY[BF16])


# ------------------------------------------------------------------ positions out of range
# the second of each: heads not made of aligned chunks, which take the plain kernels
@pytest.mark.parametrize("t,hq,hk,d,rot", [(50, 6, 2, 64, 32), (50, 3, 2, 60, 24), (3000, 8, 2, 128, 128), (9, 1, 0, 96, 96)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_positions_out_of_range_stay_with_their_tokens(oz2, t, hq, hk, d, rot, dtype, interleaved):
    q, k, dq, dk = (normal(t, h, d, dtype=dtype, seed=i) for i, h in enumerate((hq, hk, hq, hk)))
    wq, wk = 1 + 0.1 * normal(d, dtype=dtype, seed=5), 1 + 0.1 * normal(d, dtype=dtype, seed=6)
    angle = torch.arange(100, device="cuda")[:, None] * torch.linspace(0.01, 1, rot // 2, device="cuda")
    pos = torch.arange(t, device="cuda") % 100
    bad, lost = pos.clone(), [0, 3, t // 2, t - 1]
    bad[lost] = torch.tensor([-1, 100, 2**40, -2**62], device="cuda")
    ok = [i for i in range(t) if i not in lost]
    for g in (dq, dk):  # gradients of zero add nothing
        g[lost] = 0
    want = oz2.qk_norm_rope_backward(dq, dk, q, k, wq, wk, angle.cos(), angle.sin(), pos, interleaved=interleaved)
    for g in (dq, dk):
        g[lost] = float("nan")
    got = oz2.qk_norm_rope_backward(dq, dk, q, k, wq, wk, angle.cos(), angle.sin(), bad, interleaved=interleaved)
    for a, b in zip(got[:2], want[:2]):
        assert bool(a[lost].isnan().all()) and torch.equal(a[ok], b[ok])
    assert torch.equal(got[2], want[2]) and torch.equal(got[3], want[3])
    assert bool(torch.isfinite(got[2]).all())


# ------------------------------------------------------------------ what autograd is told
def test_autograd_notices_writes_to_out(oz2):
    x, w, r = normal(8, 16), normal(24, 16, seed=1), normal(8, 24, seed=2)
    q, k, g, h = normal(5, 2, 16), normal(5, 1, 16, seed=1), normal(5, 2, 16, seed=2), normal(5, 1, 16, seed=3)
    angle, pos = torch.zeros(8, 8, device="cuda"), torch.zeros(5, dtype=torch.int64, device="cuda")
    one = torch.ones(16, dtype=BF16, device="cuda")
    stream = torch.cuda.current_stream()
    for f, outs in ((lambda: oz2.linear(x, w, residual=r, out=r), (r,)), (lambda: oz2.linear(x, w, out=r, stream=stream), (r,)),
                    (lambda: oz2.dropout(x, 0.5, seed=1, out=x), (x,)), (lambda: oz2.dropout_backward(x, 0.5, seed=1, out=x), (x,)),
                    (lambda: oz2.qk_norm_rope(q, k, one, one, angle, angle, pos, out=(q, k)), (q, k)),
                    (lambda: oz2.qk_norm_rope_backward(g, h, q, k, one, one, angle, angle, pos, out=(g, h)), (g, h))):
        before = [t._version for t in outs]
        f()
        assert all(t._version > v for t, v in zip(outs, before))
    # a saved tensor that a call overwrites is refused, not used
    leaf = normal(8, 24, dtype=F32).requires_grad_(True)
    saved = leaf.to(BF16) * 2
    loss = (saved * saved).sum()
    oz2.linear(x, w, out=saved.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    # tensors made under inference mode have no version
    with torch.inference_mode():
        out = torch.empty(8, 24, dtype=BF16, device="cuda")
        oz2.linear(x, w, out=out)


# ------------------------------------------------------------------ calls that fail on the host
def test_a_failed_call_leaves_no_error_behind(oz2):
    # a launch is refused on a stream whose capture was cut short; torch and the library's other calls share the
    # runtime's record of the last error, and would report it as theirs
    from emulated_fp64_gemm_gb300.layers import _library

    runtime = _library()  # which links the shared CUDA runtime
    x, w = normal(8, 16), normal(24, 16, seed=1)
    a = torch.ones(64, 64, dtype=torch.float64, device="cuda")
    want, out = oz2.linear(x, w), torch.empty(8, 24, dtype=BF16, device="cuda")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    handle, graph = ctypes.c_void_p(stream.cuda_stream), ctypes.c_void_p()
    assert runtime.cudaStreamBeginCapture(handle, 2) == 0
    try:
        assert runtime.cudaStreamSynchronize(handle) != 0  # not permitted: it ends the capture with an error
        runtime.cudaGetLastError()
        with torch.cuda.stream(stream), pytest.raises(oz2.Ozaki2Error):
            oz2.linear(x, w, out=out)
        left = runtime.cudaPeekAtLastError()
    finally:
        runtime.cudaStreamEndCapture(handle, ctypes.byref(graph))
        runtime.cudaGetLastError()
    assert left == 0
    with torch.cuda.stream(stream):
        oz2.linear(x, w, out=out)
        oz2.dgemm(a, a, 8, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("d,rot", [(64, 32), (60, 24)])
def test_tables_without_rows(oz2, d, rot):
    # every position is outside them
    q, k, one = normal(5, 2, d), normal(5, 1, d, seed=1), torch.ones(d, dtype=BF16, device="cuda")
    empty, pos = torch.empty(0, rot // 2, device="cuda"), torch.zeros(5, dtype=torch.int64, device="cuda")
    for t in oz2.qk_norm_rope(q, k, one, one, empty, empty, pos):
        assert bool(t.isnan().all())
    dq, dk, dwq, dwk = oz2.qk_norm_rope_backward(q, k, q, k, one, one, empty, empty, pos)
    assert bool(dq.isnan().all()) and bool(dk.isnan().all()) and not dwq.any() and not dwk.any()
    assert oz2.qk_norm_rope(q[:0], k[:0], one, one, empty, empty, pos[:0])[0].shape == (0, 2, d)
