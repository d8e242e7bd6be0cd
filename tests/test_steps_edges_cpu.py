"""Host-side checks of the step operators beside those of test_steps_cpu: what a call may leave out, and what it refuses."""
import pytest

import emulated_fp64_gemm_gb300 as oz2  # noqa: F401
from emulated_fp64_gemm_gb300 import _build

torch = pytest.importorskip("torch")
from emulated_fp64_gemm_gb300 import steps  # noqa: E402
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
    assert oz2.TokenLogprobs._fields == ("logprobs", "z_max", "log_sum", "entropy", "top_logprobs", "top_ids", "lse")
    saved = oz2.TokenLogprobs(logprobs=one, lse=one, entropy=None, top_logprobs=None, top_ids=None)
    assert saved.lse is one and saved.z_max is None and saved.log_sum is None
