"""Calls captured in CUDA graphs that use the library's workspace: replayed after the
workspace has grown, and captured on streams that have none yet."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def oz2():
    import __graft_entry__ as g

    g.build()
    import emulated_fp64_gemm_gb300 as m

    assert torch.cuda.is_available()
    yield m
    torch.cuda.synchronize()
    m.workspace_release()
    assert m.last_error() == 0


def normal(*shape, dtype=BF16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 31 * sum(shape))
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def calls(oz2, scale):
    """(name, function) of calls that need a workspace; `scale` makes their sizes larger."""
    m, k, n = 70 * scale, 130 * scale, 99 * scale
    x, w, dy, z = normal(m, k, dtype=F16), normal(n, k, dtype=F16, seed=1), normal(m, n, dtype=F16, seed=2), normal(m, n, dtype=F16, seed=3)
    t = 50 * scale
    q, kk, dq, dk = normal(t, 4, 64), normal(t, 2, 64, seed=1), normal(t, 4, 64, seed=2), normal(t, 2, 64, seed=3)
    wq, wk = normal(64, seed=4), normal(64, seed=5)
    angle = torch.arange(64, device="cuda")[:, None] * torch.linspace(0.01, 1, 32, device="cuda")
    pos = torch.arange(t, device="cuda") % 64
    a, b = (torch.randn(64 * scale, 64 * scale, device="cuda", dtype=torch.float64) for _ in range(2))
    return [
        ("linear", lambda: (oz2.linear(x, w, activation="silu"),)),
        ("linear_backward", lambda: oz2.linear_backward(dy, x, w, preact=z, activation="gelu", dropout=0.25, seed=3)),
        ("qk_norm_rope_backward", lambda: oz2.qk_norm_rope_backward(dq, dk, q, kk, wq, wk, angle.cos(), angle.sin(), pos)),
        ("dgemm", lambda: (oz2.dgemm(a, b, 8),)),
    ]


def capture(oz2, f, stream):
    """A graph of f() on `stream`, and its outputs."""
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        out = f()
    return g, out


@pytest.mark.parametrize("which", range(4))
def test_replay_after_the_workspace_has_grown(oz2, which):
    stream = torch.cuda.Stream()
    name, f = calls(oz2, 1)[which]
    want = [t.clone() for t in f()]
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        f()
    stream.synchronize()
    g, out = capture(oz2, f, stream)
    # a larger call on the same stream, and memory that would take the place of what it freed
    with torch.cuda.stream(stream):
        calls(oz2, 6)[which][1]()
    stream.synchronize()
    junk = [torch.full((1 << n,), 0x7FC0, dtype=torch.int16, device="cuda") for n in range(10, 24)]
    held = [t.clone() for t in junk]
    for t in out:
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, want):
        assert torch.equal(a, b), name
    assert all(torch.equal(a, b) for a, b in zip(junk, held))
    # the stream's calls use the larger block; the graph and they keep giving the same
    with torch.cuda.stream(stream):
        again = f()
    stream.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and torch.equal(c, b) for a, b, c in zip(out, want, again))


@pytest.mark.parametrize("which", range(4))
def test_capture_on_a_stream_without_a_workspace(oz2, which):
    name, f = calls(oz2, 2)[which]
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        want = [t.clone() for t in f()]
    torch.cuda.synchronize()
    oz2.workspace_release()
    g, out = capture(oz2, f, None)
    for _ in range(2):
        for t in out:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), name


def test_a_workspace_that_grows_within_a_capture(oz2):
    small, large = calls(oz2, 1), calls(oz2, 5)
    want = [t.clone() for _, f in small + large for t in f()]
    torch.cuda.synchronize()
    oz2.workspace_release()
    g, out = capture(oz2, lambda: [t for _, f in small + large for t in f()], torch.cuda.Stream())
    for t in out:
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
