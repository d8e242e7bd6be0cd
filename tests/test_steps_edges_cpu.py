"""Host-side checks of the step operators beside those of test_steps_cpu: what a call may leave out, and what it refuses."""
import copy
import io
import os

import pytest

import emulated_fp64_gemm_gb300 as oz2  # noqa: F401
from emulated_fp64_gemm_gb300 import _build

torch = pytest.importorskip("torch")
from emulated_fp64_gemm_gb300 import steps  # noqa: E402
from tests._util import ROOT  # noqa: E402
from tests.test_steps_cpu import CUDA, INVALID, P, logprobs, logprobs_backward  # noqa: E402


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return steps._library()


# ------------------------------------------------------------------ token_logprobs
def test_lse_stands_for_both_numbers(lib):
    assert logprobs_backward(lib, z_max=0, log_sum=0) == INVALID and logprobs(lib, lse=P, log_sum=0) == INVALID
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: what follows would be enqueued")
    # past the checks, up to the missing device
    assert logprobs(lib, lse=P) == CUDA and logprobs_backward(lib, lse=P) == CUDA
    assert logprobs_backward(lib, z_max=0, log_sum=0, lse=P) == CUDA and logprobs_backward(lib, z_max=0, lse=P) == CUDA


def test_names_of_what_log_probabilities_keep():
    one = torch.zeros(1)
    assert oz2.TokenLogprobs._fields == ("logprobs", "z_max", "log_sum", "entropy", "top_logprobs", "top_ids")
    logprobs, z_max, log_sum, entropy, top_logprobs, top_ids = oz2.TokenLogprobs(*range(6), lse=7)  # six, as ever
    assert (logprobs, z_max, log_sum, entropy, top_logprobs, top_ids) == (0, 1, 2, 3, 4, 5)
    for t in (oz2.TokenLogprobs(*range(6), lse=7), oz2.TokenLogprobs(*range(6), 7)):
        assert t.lse == copy.copy(t).lse == t._replace(z_max=9).lse == 7 and t._replace(z_max=9).z_max == 9
        assert t._replace(lse=8).lse == 8 and t._replace(lse=None).lse is None and t[:4] == (0, 1, 2, 3)
    saved = oz2.TokenLogprobs(logprobs=one, lse=one, entropy=None, top_logprobs=None, top_ids=None)
    assert saved.lse is one and saved.z_max is None and saved.log_sum is None


# ------------------------------------------------------------------ adamw
def test_a_state_is_that_of_its_parameters():
    sizes = [300, 10, 5]
    for bits, master in ((32, False), (8, True)):
        state = oz2.adamw_state([torch.ones(n, dtype=torch.bfloat16) for n in sizes], bits=bits, master=master)
        copies = [state, state._replace(exp_avg=state.exp_avg.clone()), copy.copy(state), copy.deepcopy(state)]
        file = io.BytesIO()
        torch.save(state, file)
        file.seek(0)
        copies.append(torch.load(file, weights_only=False))
        for s in copies:
            assert type(s) is oz2.AdamWState and s.sizes == sizes
            assert steps._check_state(s, sizes, torch.bfloat16, -1) == bits
            # as many blocks of 256 each
            for other in ([10, 300, 5], [300, 5, 10], [301, 10, 5], [300, 10, 5, 0], [1, 1, 1, 1]):
                with pytest.raises(ValueError, match="another order"):
                    steps._check_state(s, other, torch.bfloat16, -1)
        # tensors alone: their length is known, and no more
        loose = oz2.AdamWState(*state)
        assert loose.sizes is None and steps._check_state(loose, [10, 300, 5], torch.bfloat16, -1) == bits
        with pytest.raises(ValueError):
            steps._check_state(loose, [300, 300, 5], torch.bfloat16, -1)


def test_what_is_no_tensor_is_named():
    params = [torch.ones(4), torch.ones(3)]
    state = oz2.adamw_state(params)
    for p, g, name in ((params, [torch.ones(4), None], r"grads\[1\]"), (params, [None, None], r"grads\[0\]"), ([None, params[1]], params, r"params\[0\]")):
        with pytest.raises(TypeError, match=name + " must be a tensor, got NoneType"):
            oz2.adamw(p, g, state, lr=1e-3)


# ------------------------------------------------------------------ temperatures
def test_temperatures_are_refused_by_their_bounds(lib):
    for t in (1e31, 9.9e-31, -1.0, float("inf"), float("nan")):
        assert logprobs(lib, temperature=t) == logprobs_backward(lib, temperature=t) == INVALID
        with pytest.raises(ValueError, match="between 1e-30 and 1e30"):
            steps._temperature(t)
    assert "1e-30 <= temperature <= 1e30" in open(os.path.join(ROOT, "include", "ozaki2_steps.h")).read()
    for t in (1e-30, 1, 1e30):
        assert steps._temperature(t) == t
