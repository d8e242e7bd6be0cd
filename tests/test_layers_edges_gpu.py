"""The layer operators where they leave the ordinary path: waits that run out, the ends of
the types' ranges, activations' tails, positions out of range, and what autograd is told."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


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
