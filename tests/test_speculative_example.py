"""The example's step count is bounded on the host, before anything runs on the GPU: past its rotation table and pages an
index would leave its table."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("speculative_step", os.path.join(ROOT, "examples", "speculative_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


class Started(Exception):
    pass


def test_steps_past_the_positions_are_refused(monkeypatch):
    ex = example()

    def block(batch, drafts):
        raise Started
    monkeypatch.setattr(ex, "Block", block)
    for steps in (-1, ex.MOST_STEPS + 1, 10 ** 9):
        with pytest.raises(SystemExit):
            ex.main(steps)
    for steps in (0, 8, ex.MOST_STEPS):
        with pytest.raises(Started):
            ex.main(steps)


def test_the_most_steps_fit_the_positions_and_the_pages():
    ex = example()
    for steps, fits in ((ex.MOST_STEPS, True), (ex.MOST_STEPS + 1, False)):
        # every step writes drafts + 1 places and keeps at most as many
        last = ex.PROMPT + steps * (ex.DRAFTS + 1)   # one past the last position
        assert (last <= ex.MAX_POS) == fits
    assert ex.MOST_STEPS * (ex.DRAFTS + 1) <= ex.MAX_POS // ex.PAGE * ex.PAGE
