"""The oracle's 4-bit form where a top code would not stand for a number of the type."""
import numpy as np
import pytest
import torch

from oracle import pw_context as X


def half(a):
    with np.errstate(over="ignore"):
        return np.asarray(a).astype(np.float16)


def test_the_next_lower_step_where_a_top_code_would_be_an_infinity():
    x = np.zeros((4, 32))
    x[0, 0] = 65504               # 4366.93 rounds to 4368, and 15 of it to infinity: 4364
    x[1, :2] = 65504, -65504      # 8733.87 to 8736, -65504 + 131040 = 65536: 8728
    x[2, 0] = 65472               # 4364.8 rounds to 4364
    x[3, 1:] = -65504             # downwards nothing is in the way: 4368
    c, least, step = X.quantise(x, half)
    assert step[:, 0].tolist() == [4364, 8728, 4364, 4368] and least[:, 0].tolist() == [0, -65504, 0, -65504]
    assert c[0, 0] == 15 and c[1, :3].tolist() == [15, 0, 8] and c[3, 0] == 15
    v = X.values(c, least, step)
    assert np.isfinite(half(v)).all() and v[3, 0] == 16
    bf16 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).bfloat16().float().numpy()  # noqa: E731
    x = np.full((1, 32), 8 * 2.0 ** 120)
    x[0, 3] = 255 * 2.0 ** 120    # 247 / 15 rounds to 16.5, 8 + 247.5 to 256
    c, least, step = X.quantise(x, bf16)
    assert step[0, 0] == 16.375 * 2.0 ** 120 and np.isfinite(bf16(X.values(c, least, step))).all() and c[0, 3] == 15


@pytest.mark.parametrize("seed", range(4))
def test_groups_of_finite_halves_stand_for_finite_halves(seed):
    rng = np.random.default_rng(seed)
    ends = rng.choice([0, 1, 65504, -65504, 65440, 60000, -30000], (500, 2))
    x = half(ends[:, :1] + (ends[:, 1:] - ends[:, :1]) * rng.random((500, 32)))
    x[:, :2] = ends
    c, least, step = X.quantise(x, half)
    assert np.isfinite(half(X.values(c, least, step))).all() and (half(step) == step).all()
