"""Pins of the oracle of the calls around the layer, each against a closed form or an independent computation."""
import math

import numpy as np
import pytest

from oracle import pw_serve as S


def _table(maxpos, rot):
    inv = 10000.0 ** (-np.arange(rot // 2) * 2 / rot)
    ang = np.arange(maxpos)[:, None] * inv
    return np.concatenate([np.cos(ang), np.sin(ang)], 1)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [0, 4, 8])
def test_rotation_is_a_complex_product_and_keeps_relative_positions(inter, rot):
    rng = np.random.default_rng(1)
    x, y = rng.standard_normal((2, 3, 2, 8))
    tab = _table(50, rot) if rot else None
    pos = [0, 3, 41]
    a = S.norm_rope(x, None, 0.0, tab, pos, inter)
    assert np.allclose(a[0], x[0])                                      # position 0 turns nothing
    assert np.allclose((a ** 2).sum(-1), (x ** 2).sum(-1))              # lengths stay
    assert np.array_equal(a[..., rot:], x[..., rot:])
    b = S.norm_rope(y, None, 0.0, tab, pos, inter)
    a2 = S.norm_rope(x, None, 0.0, tab, [7, 10, 48], inter)
    b2 = S.norm_rope(y, None, 0.0, tab, [7, 10, 48], inter)
    assert np.allclose((a * b).sum(-1), (a2 * b2).sum(-1))              # a common shift of positions changes no product
    for i in range(rot // 2):
        ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
        z = (x[..., ia] + 1j * x[..., ib]) * np.array([complex(tab[p, i], tab[p, rot // 2 + i]) for p in pos])[:, None]
        assert np.allclose(a[..., ia], z.real) and np.allclose(a[..., ib], z.imag)


def test_norm_has_unit_mean_square_before_the_weight():
    x = np.random.default_rng(2).standard_normal((2, 3, 16)) * 7
    assert np.allclose((S.norm_rope(x, np.ones(16), 0.0, None, None, False) ** 2).mean(-1), 1)
    w = np.arange(16.0)
    assert np.allclose(S.norm_rope(x, w, 0.0, None, None, False), S.norm_rope(x, np.ones(16), 0.0, None, None, False) * w)
    assert np.allclose(S.norm_rope(np.full((1, 1, 4), 3.0), np.ones(4), 7.0, None, None, False), 3 / 4)


def test_append_writes_its_slots_and_nothing_else():
    c = np.zeros((3, 2, 4, 2))
    rows = np.arange(12.0).reshape(3, 2, 2) + 1
    d = S.append(c, rows, [5, -1, 12])
    assert np.array_equal(d[1, :, 1], rows[0])
    assert (d != 0).sum() == 4


def test_attention_closed_forms():
    D, page = 4, 2
    kc, vc = np.zeros((4, 1, page, D)), np.random.default_rng(3).standard_normal((4, 1, page, D))
    q = np.ones((2, 1, D))
    table, ptab = np.array([[2, 1], [3, 0]]), np.array([[1, 0]])
    # equal scores: the mean of what is seen, lse = ln n
    out, lse, _, _, n = S.attend(q, kc, vc, table, [3, 0], 1, 1.0, ptab, [1], None)
    seen = np.stack([vc[1, 0, 0], vc[2, 0, 0], vc[2, 0, 1], vc[1, 0, 0]])
    assert np.allclose(out[0, 0], seen.mean(0)) and math.isclose(lse[0, 0], math.log(4))
    assert np.allclose(out[1, 0], vc[1, 0, 0]) and n[1, 0] == 1
    # nothing seen
    out, lse, *_ = S.attend(q, kc, vc, table, [0, 0], 1, 1.0)
    assert not out.any() and np.isneginf(lse).all()
    # causal among the query tokens: query j of 2 sees len - 1 + j keys
    out, lse, _, _, n = S.attend(q, kc, vc, table[:1], [2], 2, 1.0)
    assert n[:, 0].tolist() == [1, 2] and np.allclose(out[0, 0], vc[2, 0, 0])
    # one key ahead of the others by a huge margin takes everything
    kc[2, 0, 1] = 100
    out, lse, *_ = S.attend(q[:1], kc, vc, table[:1], [3], 1, 1.0)
    assert np.allclose(out[0, 0], vc[2, 0, 1]) and math.isclose(lse[0, 0], 400)


def test_a_prefix_is_the_same_as_its_tokens_in_front_of_the_suffix():
    rng = np.random.default_rng(4)
    kc, vc = rng.standard_normal((2, 8, 2, 2, 4))
    q = rng.standard_normal((2, 4, 4))
    a = S.attend(q, kc, vc, np.array([[4, 5]]), [3], 2, 0.5, np.array([[1, 2]]), [4])
    b = S.attend(q, kc, vc, np.array([[1, 2, 4, 5]]), [7], 2, 0.5)
    assert np.allclose(a[0], b[0]) and np.allclose(a[1], b[1])


def test_verification_by_hand():
    p = np.array([[[.5, .25, .25], [.1, .6, .3], [.2, .3, .5]]], dtype=np.float32)
    q = np.array([[[.9, .05, .05], [.2, .2, .6]]], dtype=np.float32)
    e = np.ones((1, 3), dtype=np.float32)
    tok = np.array([[0, 2]])
    # .5 * .9 < .5 keeps token 0; .6 * .6 < .3 does not keep token 2: residual (0, .4, 0)
    out, a = S.verify(p, q, tok, [2], np.array([[.5, .6]]), e)
    assert a.tolist() == [1] and out.tolist() == [[0, 1, -1]]
    out, a = S.verify(p, q, tok, [2], np.array([[.5, .4]]), e)   # all kept: the next from p_2
    assert a.tolist() == [2] and out.tolist() == [[0, 2, 2]]
    out, a = S.verify(p, q, tok, [0], np.array([[.5, .4]]), e)   # no drafts: from p_0
    assert a.tolist() == [0] and out.tolist() == [[0, -1, -1]]
    out, a = S.verify(p, p[:, :2].copy() * 2, tok, [2], np.array([[.9, .9]]), e)  # refused, residual all zero: from p_0
    assert out.tolist() == [[0, -1, -1]]


def test_verified_tokens_follow_the_target_distribution():
    rng = np.random.default_rng(5)
    n, V = 20000, 4
    pt = np.array([.4, .3, .2, .1], dtype=np.float32)
    qd = np.array([.1, .2, .3, .4], dtype=np.float32)
    tok = rng.choice(V, size=(n, 1), p=qd / qd.sum())
    out, _ = S.verify(np.tile(pt, (n, 2, 1)), np.tile(qd, (n, 1, 1)), tok, np.ones(n), rng.random((n, 1)),
                      rng.exponential(size=(n, V)).astype(np.float32))
    freq = np.bincount(out[:, 0], minlength=V) / n
    assert np.abs(freq - pt).max() < 5 * math.sqrt(.25 / n)  # five standard deviations
