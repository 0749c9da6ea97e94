"""Host side of the calls of test_context_host that came behind them, without a GPU (host-simulated device)."""
import pytest

import any_precision_expert_gb300 as pw
from any_precision_expert_gb300._lib import lib

UNSUPPORTED = 2


@pytest.fixture(autouse=True)
def sim():
    lib.pw_testing_host_sim(1)
    yield
    lib.pw_testing_host_sim(0)


def test_prompt_error_word_needs_a_device():
    assert lib.pw_prompt_check_device(None) == UNSUPPORTED and pw.prompt_check_device() == UNSUPPORTED
