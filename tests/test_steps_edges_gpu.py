"""The step operators where they leave the ordinary path: what may be kept between a pass and its gradient, codes at
ties, rows that share blocks, confident rows, crowded alternatives and long steps."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
from tests import _steps_ref as ref  # noqa: E402
from tests._layers_ref import TINY, UNIT, assert_within  # noqa: E402
from tests.test_steps_gpu import check_norm, check_step, generator, normal, some_targets, strided, tensors, values  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, F16, F32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def oz2():
    import __graft_entry__ as g

    g.build()
    import emulated_fp64_gemm_gb300 as m

    assert torch.cuda.is_available()
    yield m
    assert m.last_error() == 0


# ------------------------------------------------------------------ one number per row between the passes
@pytest.mark.parametrize("rows,vocab", [(3, 9), (7, 1000), (4, 20001), (2, 131072), (1300, 700)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_gradient_from_lse_alone(oz2, rows, vocab, dtype):
    """lse is off by a sum of vocab exponentials (see test_steps_gpu) and roundings of z_max's and its own size, 2^-22 of
    them; log p = z - lse then by that and 2^-22 |z| once more (e), p by a factor 1 + e, p (log p + H) by p e (2 + |log p| + H)."""
    for temperature, entropy in ((1.0, True), (0.7, False), (1.3, True)):
        logits, targets = normal(rows, vocab, dtype=dtype, scale=3.0), some_targets(rows, vocab)
        logits[0, ::2] = -INF
        got = oz2.token_logprobs(logits, targets, temperature=temperature, entropy=entropy)
        z_max, log_sum, _, ent, logp = ref.token_logprobs(logits, targets, temperature, -100)
        lse = z_max + log_sum
        rel = (vocab / 64 + 64) * 2.0**-24 + 2.0**-21
        off = rel * (1 + log_sum) + 2.0**-22 * (z_max.abs() + lse.abs())
        assert_within(got.lse, lse, off, "lse")
        g, h = normal(rows, seed=5), normal(rows, seed=6) if entropy else None
        saved = oz2.TokenLogprobs(logprobs=got.logprobs, lse=got.lse, entropy=got.entropy)
        d = oz2.token_logprobs_backward(g, logits, targets, saved, dentropy=h, temperature=temperature)
        p, known = torch.exp(logp), targets != -100
        gd = torch.where(known, g.double(), 0.0)[:, None]
        onehot = torch.zeros_like(p).scatter_(1, targets.clamp(min=0)[:, None], 1.0) * known[:, None]
        near = logp.clamp(min=-200)
        # (the target's own element comes from its log p, which keeps its precision)
        at_target = -torch.expm1(torch.where(torch.isfinite(logp), logp, -1e300))
        want = torch.where(onehot > 0, gd * at_target, -gd * p)
        e = off[:, None] + 2.0**-22 * (near.abs() + lse.abs()[:, None]) + 2.0**-20
        err = gd.abs() * torch.where(onehot > 0, at_target, p) * e
        if entropy:
            want = want - h.double()[:, None] * p * (near + ent[:, None])
            err = err + h.double().abs()[:, None] * p * e * (2 + near.abs() + ent[:, None])
        err = (2 * err + 2.0**-120) / temperature
        assert_within(d, want / temperature, err + UNIT[dtype] * (want.abs() / temperature + err) + TINY[dtype], "dlogits")
    # beside both numbers lse is not read
    saved = got._replace(lse=torch.full_like(got.lse, NAN))
    again = oz2.token_logprobs_backward(g, logits, targets, got, dentropy=h, temperature=temperature)
    assert torch.equal(oz2.token_logprobs_backward(g, logits, targets, saved, dentropy=h, temperature=temperature), again)


def test_lse_of_special_rows(oz2):
    x = normal(5, 3000, dtype=F32)
    x[0], x[1, 7], x[2, 8] = -INF, NAN, INF
    x[3] = -3e38
    targets = torch.zeros(5, dtype=torch.int64, device="cuda")
    got = oz2.token_logprobs(x, targets, temperature=0.5)
    assert got.lse[0] == got.lse[3] == -INF and bool(got.lse[1:3].isnan().all()) and bool(torch.isfinite(got.lse[4]))
    saved = oz2.TokenLogprobs(logprobs=got.logprobs, lse=got.lse)
    d = oz2.token_logprobs_backward(torch.ones(5, device="cuda"), x, targets, saved, temperature=0.5)
    assert not d[[0, 3]].any() and bool(d[1:3].isnan().all()) and bool(torch.isfinite(d[4]).all())
    for saved in (oz2.TokenLogprobs(got.logprobs), got._replace(z_max=None, lse=None), got._replace(log_sum=None, lse=None)):
        with pytest.raises(ValueError, match="lse"):
            oz2.token_logprobs_backward(torch.ones(5, device="cuda"), x, targets, saved)
    with pytest.raises(ValueError):
        oz2.token_logprobs_backward(torch.ones(5, device="cuda"), x, targets, oz2.TokenLogprobs(got.logprobs, lse=got.lse[:2]))


# ------------------------------------------------------------------ 8-bit codes
TIES = torch.tensor((ref.E4M3[:126] + ref.E4M3[1:127]) / 2, dtype=torch.float64)


def weights_at_ties(cols, width, dtype):
    """Weights of which each `width` have a largest one T and, for the others, products of T / 448 with the midpoints of
    neighbouring codes, and what lies up to three 32-bit steps beside them (less, where the type has fewer bits)."""
    rng = np.random.default_rng(cols)
    w = np.zeros(cols, np.float32)
    for at in range(0, cols, width):
        n = min(width, cols - at)
        # (a largest one of few bits in 16 bits: three quarters of its multiples are ties' products, to the bit)
        top = np.float32(rng.uniform(1, 2)) if dtype is F32 else np.float32(rng.choice([1.3125, 1.5, 1.125, 1.6875]))
        scale = top / np.float32(448)
        near = (rng.choice(TIES.numpy(), n) * np.float64(scale)).astype(np.float32)
        if dtype is F32:
            near = (near.view(np.int32) + rng.integers(-3, 4, n).astype(np.int32)).view(np.float32)
        w[at:at + n] = near
        w[at + rng.integers(n)] = 0.0  # of both signs in the rows
        w[at + rng.integers(n)] = top
    return torch.from_numpy(w).cuda().to(dtype)


def exactly_one(n):
    return np.float32(n) * np.float32(1 / n) == 1


@pytest.mark.parametrize("cols", [c for c in (128, 1024, 1003, 4096, 5001, 8200, 16384, 20000, 20002) if exactly_one(c)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("block", [None, 128])
def test_codes_are_those_of_the_quotient(oz2, cols, dtype, block):
    """Rows of 1 and -1 have the norm 1, so that y is the weight to the bit, scale its largest magnitude over 448 and each
    code y / scale, both rounded to 32 bits, rounded once: a tie goes to the even code, its neighbours to theirs."""
    w = weights_at_ties(cols, block or cols, dtype)
    for rows in (3, 700):
        x = torch.where(normal(rows, cols) < 0, -1.0, 1.0).to(dtype)
        y = oz2.rms_norm(x, w, eps=0.0)
        assert torch.equal(y, x * w)
        for residual in (None, torch.zeros_like(x)):
            q, scale = oz2.rms_norm(x, w, residual=residual, eps=0.0, out_dtype=E4M3, block=block)[:2]
            exact = y.float().cpu().numpy()
            width = block or cols
            tops = np.stack([np.abs(exact[:, at:at + width]).max(1) for at in range(0, cols, width)], 1)
            want = tops / np.float32(448)
            assert np.array_equal(scale.cpu().numpy(), want)
            codes = ref.to_e4m3((exact / want.repeat(width, 1)[:, :cols]).ravel()).reshape(rows, cols)
            got = q.view(torch.uint8).cpu().numpy()
            assert np.array_equal(got, codes), int((got != codes).sum())


@pytest.mark.parametrize("cols", [200, 2048, 1003, 9000, 20000])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size,weight", [(1e10, 1e30), (1e18, 1e21), (1e-14, 1e-29), (1e-9, 1e-34), (1e30, 1e-25), (1e-30, 1e25)])
def test_codes_of_products_out_of_range(oz2, cols, dtype, size, weight):
    # x times the weight leaves the 32-bit range, x over its norm times the weight does not
    x, w = normal(7, cols, dtype=dtype, scale=size), normal(cols, dtype=dtype, scale=weight, seed=1)
    x[2] = 0
    for residual in (None, torch.zeros_like(x)):
        for block in (None, 128):
            x[2, 0] = 0
            check_norm(oz2, x, w, residual, eps=1e-38, quantize=True, block=block)


# ------------------------------------------------------------------ token_logprobs
@pytest.mark.parametrize("vocab", [10, 5003, 131072])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("temperature", [1.0, 0.7])
def test_entropy_gradient_of_confident_rows(oz2, vocab, dtype, temperature):
    """Where one token has almost all of the probability, its element is -h p (log p + H), which is far smaller than z_max:
    log p and H are each off by a factor (see test_logprobs_of_confident_rows), H is more than eight times -log p, and the
    others' p and log p by 2^-22 of z's size: 2^-13 of every element in all, beside the output's rounding."""
    gaps = torch.tensor([10.0, 14.0, 20.0, 30.0, 40.0, 60.0], device="cuda") * temperature
    at = torch.tensor([0, vocab // 2, vocab - 1, 3, 5, 1], device="cuda")
    logits = (normal(6, vocab) * 0.5).to(dtype).float()
    logits.scatter_(1, at[:, None], (gaps + math.log(vocab)).to(dtype).float()[:, None])
    logits = logits.to(dtype)
    h = normal(6, seed=3) + 300.0
    for targets, g in ((torch.full_like(at, -100), normal(6, seed=4)), ((at + 1) % vocab, torch.zeros(6, device="cuda"))):
        saved = oz2.token_logprobs(logits, targets, temperature=temperature, entropy=True)
        got = oz2.token_logprobs_backward(g, logits, targets, saved, dentropy=h, temperature=temperature)
        z = logits.double() / temperature
        d = z - z.gather(1, at[:, None])
        others = torch.exp(d).scatter(1, at[:, None], 0.0)
        rho, bent = others.sum(1, keepdim=True), -(others * d).sum(1, keepdim=True)
        # log p + H = d + bent / (1 + rho): nothing of it is a difference of larger numbers
        want = -h.double()[:, None] * torch.exp(d) / (1 + rho) * (d + bent / (1 + rho)) / temperature
        assert_within(got, want, 2.0**-13 * want.abs() + UNIT[dtype] * (1 + 2.0**-13) * want.abs() + TINY[dtype])


def test_nan_at_the_first_place_of_crowded_rows(oz2):
    # more large logits in the reach of 31 groups of threads than there is room for, and a NaN before them
    vocab, rows = 262144, 400
    columns = torch.arange(vocab, device="cuda")
    logits = normal(rows, vocab, scale=0.1)
    some = columns % 2048 < 992
    logits[::40] = torch.where(some, 5 + torch.rand(vocab, generator=generator(1), device="cuda"), logits[::40])
    logits[0, 0] = logits[40, 0] = logits[40, 77] = logits[80, 8] = NAN
    order = torch.sort(logits[::40].nan_to_num(100.0), dim=-1, descending=True, stable=True).indices[:, :32]
    got = oz2.token_logprobs(logits, torch.zeros(rows, dtype=torch.int64, device="cuda"), top=32)
    assert torch.equal(got.top_ids[::40], order)
    assert got.top_ids[0, 0] == 0 and got.top_ids[40, :2].tolist() == [0, 77] and got.top_ids[80, 0] == 8
    assert bool(got.top_logprobs[[0, 40, 80]].isnan().all()) and bool(torch.isfinite(got.top_logprobs[120]).all())


def test_adamw_refuses_the_state_of_other_parameters(oz2):
    params, grads = tensors([300, 10], BF16, F32)
    state = oz2.adamw_state(params, bits=8, master=True)
    before = [t.clone() for t in (*params, *state)]
    with pytest.raises(ValueError, match="another order"):
        oz2.adamw(params[::-1], grads[::-1], state, lr=1e-3)
    for a, b in zip((*params, *state), before):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    check_step(oz2, params, grads, state)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("entropy", [False, True])
def test_gradient_of_masked_targets(oz2, dtype, entropy):
    # a target that is masked has log p -inf, whose gradient is that of probability 0; no other masked logit has one
    for vocab, temperature in ((9, 1.0), (3001, 0.5)):
        logits = normal(4, vocab, dtype=dtype)
        logits[:3, ::2] = -INF
        logits[3] = -INF
        targets = torch.tensor([2, 1, -100, 4], device="cuda")
        saved = oz2.token_logprobs(logits, targets, temperature=temperature, entropy=entropy)
        assert saved.logprobs[0] == saved.logprobs[3] == -INF
        g = torch.full((4,), 3.0, device="cuda")
        d = oz2.token_logprobs_backward(g, logits, targets, saved, dentropy=g if entropy else None, temperature=temperature)
        assert d[0, 2] == 3.0 / temperature
        d[0, 2] = 0
        assert not d[:, ::2].any() and not d[3].any() and bool(d[:2, 1::2].all())


@pytest.mark.parametrize("vocab", [40, 5000, 70000])
def test_alternatives_fall_by_their_logits(oz2, vocab):
    """Also where the temperature, or the sum of a row, leaves nothing of the difference: -3e38 / 0.5 is masked like -inf,
    and logits of 2^-24 and less beside 1 have one log p."""
    logits = torch.full((3, vocab), -INF, device="cuda")
    logits[0, 7::3] = -3e38
    logits[0, 5] = 1.0
    logits[1, 9::2] = -3.2e38
    logits[1, 30] = -3.1e38
    logits[2] = 1.0
    logits[2, ::2] = torch.arange((vocab + 1) // 2, device="cuda") * 2.0**-149
    targets = torch.zeros(3, dtype=torch.int64, device="cuda")
    for top in (1, 9, 32):
        got = oz2.token_logprobs(logits, targets, temperature=0.5, top=top)
        want = torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, :top]
        assert torch.equal(got.top_ids, want)
        assert got.top_logprobs[0, 0] == 0 and bool((got.top_logprobs[0, 1:] == -INF).all() & (got.top_logprobs[1] == -INF).all())


# ------------------------------------------------------------------ rows that share blocks
# rows enough for every choice of warps per row and rows per run, a number that no run divides
MANY_ROWS = [(9001, 128), (5003, 1024), (5003, 2048), (2731, 4096), (1307, 8192), (1409, 8200), (1003, 10240), (701, 10240), (1103, 12288),
             (709, 16384)]


@pytest.mark.parametrize("rows,cols", MANY_ROWS)
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_norm_of_many_aligned_rows(oz2, rows, cols, dtype):
    x, r, w = normal(rows, cols, dtype=dtype), normal(rows, cols, dtype=dtype, seed=1), normal(cols, dtype=dtype, seed=2)
    # rows unlike each other, so that one in the place of another shows
    x *= torch.logspace(-2, 2, rows, base=2, device="cuda")[:, None].to(dtype)
    plain, = check_norm(oz2, x, w)
    y, s = check_norm(oz2, x, w, r)
    for block in (None, 128):
        check_norm(oz2, x, w, quantize=True, block=block)
        check_norm(oz2, x, w, r, quantize=True, block=block)
    over, res = x.clone(), r.clone()
    got = oz2.rms_norm(over, w, residual=res, out=over, residual_out=res)
    assert got[0] is over and got[1] is res and torch.equal(over, y) and torch.equal(res, s)
    over = x.clone()
    assert torch.equal(oz2.rms_norm(over, w, out=over), plain)


@pytest.mark.parametrize("rows,cols", [(1409, 8200), (1003, 10240), (701, 12288), (305, 16384), (4001, 1000)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_gradient_of_many_aligned_rows(oz2, rows, cols, dtype):
    """Sums of cols products are off by 2^-17 of their magnitudes (as in test_steps_gpu), those of `rows` parts by 2^-16."""
    x, dy, ds, w = (normal(rows, cols, dtype=dtype, seed=i) for i in range(4))
    w = w[0]
    u, tiny = UNIT[dtype], TINY[dtype]
    for d in (None, ds):
        dx, dw = oz2.rms_norm_backward(dy, x, w, dresidual=d)
        wdx, wdw, size, wsize = ref.rms_norm_backward(dy.double(), x.double(), w.double(), None if d is None else d.double(), 1e-6)
        err = 2.0**-15 * size
        assert_within(dx, wdx, err + u * (wdx.abs() + err) + tiny, "dx")
        err = 2.0**-16 * wsize
        assert_within(dw, wdw, err + u * (wdw.abs() + err) + tiny, "dw")
        over = dy.clone()
        assert torch.equal(oz2.rms_norm_backward(over, x, w, dresidual=d, out=over)[0], dx)


# ------------------------------------------------------------------ adamw
@pytest.mark.parametrize("dtype,grad_dtype,master", [(BF16, BF16, False), (F16, F32, True)])
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("sizes", [[1_500_000, 7, 900_001], [3_000_003, 12_345, 4_000_000]])
def test_adamw_of_long_tensors(oz2, dtype, grad_dtype, master, bits, sizes):
    # several blocks of 256 elements per warp: 8-bit states to the bit over steps
    params, _ = tensors(sizes, dtype, grad_dtype)
    state = oz2.adamw_state(params, bits=bits, master=master)
    for step in range(2):
        check_step(oz2, params, tensors(sizes, dtype, grad_dtype, seed=1000 * step)[1], state, seed=99)


@pytest.mark.parametrize("count", [24, 25, 128, 160, 880, 881])
def test_adamw_of_as_many_tensors_as_a_launch_takes(oz2, count):
    sizes = [1 + (i * 37) % 600 for i in range(count)]
    params, _ = tensors(sizes, BF16, BF16)
    state = oz2.adamw_state(params, bits=8)
    for step in range(2):
        check_step(oz2, params, tensors(sizes, BF16, BF16, seed=1000 * step)[1], state, seed=5)


@pytest.mark.parametrize("cols", [256, 1003, 2048, 20000])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_codes_beside_an_infinite_one(oz2, cols, dtype):
    # an element over the norm times its weight is past the 32-bit range: its block's scale is infinite and stands for
    # 0 where y is finite (y / scale), itself for NaN
    x, w = normal(5, cols, dtype=dtype), normal(cols, dtype=dtype, seed=1)
    x[2, 100], w[100] = 50.0, 3e38
    x[[0, 1, 3, 4], 100] = 0
    for residual in (None, torch.zeros_like(x)):
        for block in (None, 128):
            q, scale = oz2.rms_norm(x, w, residual=residual, out_dtype=E4M3, block=block)[:2]
            v, width = values(q), block or cols
            assert scale[2, 0] == INF and bool(v[2, 100].isnan())
            v[2, 100] = 0
            assert not v[2, :width].any()
            assert bool(torch.isfinite(scale[[0, 1, 3, 4]]).all()) and bool(torch.isfinite(scale[2, 1:]).all())
            assert bool(torch.isfinite(v).all()) and (block is None or bool(v[2, 128:].abs().sum() > 0))
