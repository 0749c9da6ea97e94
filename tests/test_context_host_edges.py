"""Host side of the calls of test_context_host that came behind them, without a GPU (host-simulated device)."""
import types

import pytest
import torch

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


@pytest.mark.parametrize("make", [lambda: pw.KvCache(torch.zeros(4, 2, 16, 64, dtype=torch.float16), torch.zeros(4, 2, 16, 64, dtype=torch.float16), 4),
                                  lambda: pw.KvCache4.empty(4, 4, 2, 16, 64, device="cpu")])
def test_a_cache_is_asked_on_its_own_device(make, monkeypatch):
    """The error word is read on a stream of the cache's device, and scratch is sized by that device's SMs, whichever device
    is the current one (a stand-in for a cache on a second GPU notes which device was current in each call)."""
    kv, calls, current = make(), [], ["cuda:0"]
    kv.k = types.SimpleNamespace(is_cuda=True, device="cuda:1")

    class Device:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            self.was, current[0] = current[0], self.d

        def __exit__(self, *a):
            current[0] = self.was

    class Lib:
        def __getattr__(self, name):
            f = getattr(lib, name)

            def call(*a):
                calls.append((name, current[0]))
                return f(*a)
            return call

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(pw.serve, "lib", Lib())
    monkeypatch.setattr(pw.serve, "_s", lambda s: calls.append(("stream", current[0])))
    assert kv.check_device() == UNSUPPORTED and kv.attend_workspace_size(3) > 0
    assert [d for _, d in calls] == ["cuda:1"] * 3 and current == ["cuda:0"], calls
