"""Pins of the oracle of prompts, scores and eviction, each against a closed form or an independent computation."""
import math

import numpy as np
import pytest

from oracle import pw_context as X
from oracle import pw_serve as S


def test_prompt_is_the_cached_attention_of_every_position():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((7, 4, 8)), rng.standard_normal((7, 2, 8)), rng.standard_normal((7, 2, 8))
    out, lse, A, ds, n = X.prompt(q, k, v, [1, 1, 5, 6], 0.7)
    assert np.isnan(out[[0, 6]]).all() and np.isnan(lse[[0, 6]]).all()
    # the same through a cache of one page: sequence 1 has rows 1..4, each the last query of its own length
    kc, vc = np.zeros((1, 2, 8, 8)), np.zeros((1, 2, 8, 8))
    kc[0, :, :4], vc[0, :, :4] = k[1:5].transpose(1, 0, 2), v[1:5].transpose(1, 0, 2)
    for i in range(4):
        o, l, a, d, s = S.attend(q[1 + i:2 + i], kc, vc, np.zeros((1, 1), int), [i + 1], 1, 0.7)
        for x, y in ((o, out), (l, lse), (a, A), (d, ds), (s, n)):
            assert np.allclose(x[0], y[1 + i])
    assert np.allclose(out[5], np.repeat(v[5], 2, axis=0))  # one row sees itself


def test_logprobs_closed_forms():
    lp, ent, ids, tops = X.logprobs(np.zeros((1, 8)), [3], 3)
    assert np.isclose(lp[0], -math.log(8)) and np.isclose(ent[0], math.log(8))
    assert ids.tolist() == [[0, 1, 2]] and np.allclose(tops, -math.log(8))
    x = np.array([[math.log(0.5), math.log(0.25), -np.inf, math.log(0.25)]])
    lp, ent, ids, tops = X.logprobs(x + 11, [2], 4)
    assert np.isneginf(lp[0]) and np.isclose(ent[0], 1.5 * math.log(2))
    assert ids.tolist() == [[0, 1, 3, -1]] and np.allclose(tops[0, :3], [math.log(0.5), math.log(0.25), math.log(0.25)])
    lp, ent, ids, _ = X.logprobs(np.array([[-np.inf] * 3, [1.0, np.nan, 2.0], [1.0, np.inf, 2.0]]), [0, -1, 9], 2)
    assert np.isneginf(lp[0]) and ent[0] == 0 and (ids[0] == -1).all()
    assert lp[1] == 0 and np.isnan(ent[1]) and ids[1].tolist() == [2, 0]
    assert np.isnan(lp[2]) and np.isnan(ent[2]) and ids[2].tolist() == [1, 2]


def test_four_bits_end_points_halves_and_bad_groups():
    half = lambda a: a.astype(np.float16)  # noqa: E731
    x = np.zeros((3, 64))
    x[0, :32] = np.arange(32) / 2.0          # 0 .. 15.5
    x[0, 0], x[0, 31] = 0.0, 15.0            # step 1
    c, least, step = X.quantise(x, half)
    assert step[0, 0] == 1 and least[0, 0] == 0
    assert c[0, 1] == 0 and c[0, 2] == 1 and c[0, 3] == 2 and c[0, 5] == 2 and c[0, 31] == 15  # halves go to even codes
    assert (X.values(c, least, step)[0, 32:] == 0).all() and step[0, 1] == 0
    x[1, 3], x[2, 40] = np.nan, np.inf
    c, least, step = X.quantise(x, half)
    v = X.values(c, least, step)
    assert np.isnan(v[1, :32]).all() and not np.isnan(v[1, 32:]).any() and np.isnan(v[2, 32:]).all()
    r = np.random.default_rng(1).standard_normal((50, 64)).astype(np.float16)
    c, least, step = X.quantise(r, half)
    err = np.abs(X.values(c, least, step) - r).reshape(50, 2, 32)
    # half a step, and where rounding has shortened the step its 15 halves
    assert (err <= step[..., None] * (0.5 + 15 * 2.0 ** -11) + 1e-7).all() and (c.reshape(50, 2, 32).min(-1) == 0).all()


def test_weights_add_up_to_the_queries():
    rng = np.random.default_rng(2)
    q, kc = rng.standard_normal((3, 4, 8)), rng.standard_normal((5, 2, 4, 8))
    table, lens = np.array([[4, 0], [1, 2], [3, 3]]), [6, 0, 1]
    _, lse, _, _, _ = S.attend(q, kc, kc, table, lens, 1, 0.5)
    out, _ = X.weigh(q, kc, table, lens, lse, np.zeros((3, 8)), 1, 0.5, 1.0)
    assert np.allclose(out.sum(1), [4, 0, 4]) and (out[0, 6:] == 0).all()  # every head's weights sum to 1
    again, _ = X.weigh(q, kc, table, lens, lse, out + 1, 1, 0.5, 0.25)
    assert np.allclose(again[0, :6], out[0, :6] * 1.25 + 0.25) and again[0, 7] == 1


@pytest.mark.parametrize("mass,n,budget,recent,want", [
    ([5, 1, 4, 1, 3], 5, 3, 1, [0, 2, 4]), ([1, 1, 1, 1, 1], 5, 3, 1, [0, 1, 4]), ([1, 1, 1, 1, 1], 5, 3, 0, [0, 1, 2]),
    ([0, 9, 0, 9, 0], 5, 2, 9, [3, 4]), ([0, 9, 0], 3, 7, 1, [0, 1, 2]), ([float("nan"), 0, -1, 2], 4, 2, 0, [1, 3]),
    ([float("nan"), float("-inf")], 2, 1, 0, [1]), ([0.0, -0.0, 0.0], 3, 2, 0, [0, 1]), ([], 0, 4, 2, [])])
def test_who_stays(mass, n, budget, recent, want):
    assert X.stays(np.array(mass, dtype=np.float32), n, budget, recent) == want


def test_evict_moves_rows_in_order():
    kc = np.arange(4 * 2.0 * 3).reshape(4, 1, 2, 3)
    mass = np.array([[1, 5, 2, 7]], dtype=np.float32)
    for new in ([[2, 0]], [[1]]):
        k, v, lens, m, kept = X.evict(kc, -kc, np.array([[2, 0]]), [4], mass, 2, 0, np.array(new))
        p = new[0][0]
        assert kept.tolist() == [[1, 3]] and lens.tolist() == [2] and m.tolist() == [[5, 7, 0, 0]]
        assert np.array_equal(k[p, 0], [kc[2, 0, 1], kc[0, 0, 1]]) and np.array_equal(v[p], -k[p])
        assert (k != kc).any(axis=(1, 2, 3)).sum() == 1
