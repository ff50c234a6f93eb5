"""Pins of the f64 oracle of the rotary and paged-cache calls: closed forms and brute force."""
import math

import numpy as np
import pytest

from oracle import kv as okv


def test_plain_frequencies_and_table():
    f = okv.frequencies(4, 10000.0)
    assert np.allclose(f, [1.0, 0.01], rtol=1e-15)
    t = okv.table(3, 4, 10000.0)
    assert np.allclose(t[2], [[math.cos(2), math.sin(2)], [math.cos(.02), math.sin(.02)]])


def test_scaled_frequencies():
    rot, base = 64, 10000.0
    f = okv.frequencies(rot, base)
    assert np.allclose(okv.frequencies(rot, base, okv.LINEAR, 4.0), f / 4)
    ntk = okv.frequencies(rot, base, okv.NTK, 4.0)
    assert ntk[0] == 1.0 and np.isclose(ntk[-1], f[-1] / 4)  # the slowest turns by 1/factor
    for kind in (okv.YARN, okv.BANDS):
        g = okv.frequencies(rot, base, kind, 8.0, low=1.0, high=4.0, original=2048)
        assert g[0] == f[0] and np.isclose(g[-1], f[-1] / 8)
        assert (g <= f * (1 + 1e-12)).all() and (g >= f / 8 * (1 - 1e-12)).all()
        assert (np.diff(g) < 0).all()


@pytest.mark.parametrize("flags", [0, okv.INTERLEAVED])
def test_rotation_is_orthogonal_and_its_transpose_is_its_inverse(flags):
    g = np.random.default_rng(1)
    x = g.standard_normal((5, 3, 12))
    cs = okv.table(40, 8, 100.0)[[0, 3, 9, 20, 39]]
    y, _ = okv.rotate(x, cs, 8, flags)
    assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))
    assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 8:], x[..., 8:])
    back, _ = okv.rotate(y, cs, 8, flags | okv.TRANSPOSE)
    assert np.allclose(back, x)


def test_rotation_layouts_are_a_permutation_of_one_another():
    g = np.random.default_rng(2)
    x = g.standard_normal((4, 2, 8))
    cs = okv.table(10, 8, 50.0)[[1, 2, 5, 9]]
    perm = [0, 2, 4, 6, 1, 3, 5, 7]  # interleaved -> half
    a, _ = okv.rotate(x, cs, 8, okv.INTERLEAVED)
    b, _ = okv.rotate(x[..., perm], cs, 8)
    assert np.allclose(a[..., perm], b)


def test_scores_depend_on_distance_alone():
    g = np.random.default_rng(3)
    q, k = g.standard_normal((2, 1, 1, 16))
    t = okv.table(100, 16, 1000.0)
    dot = [float((okv.rotate(q, t[[i]], 16)[0] * okv.rotate(k, t[[j]], 16)[0]).sum())
           for i, j in ((5, 2), (50, 47), (99, 96))]
    assert np.allclose(dot, dot[0])


def test_attention_against_brute_force():
    g = np.random.default_rng(4)
    k, v = g.standard_normal((2, 3, 2, 4, 6))
    pages = np.array([[2, 0], [1, -1]], np.int32)
    q = g.standard_normal((2, 4, 6))
    r = okv.attention(q, k, v, pages, [7, 0], 0.5)
    for h in range(4):
        rows = [(2, 0), (2, 1), (2, 2), (2, 3), (0, 0), (0, 1), (0, 2)]
        w = [math.exp(0.5 * float(q[0, h] @ k[p, h // 2, i])) for p, i in rows]
        o = sum(x * v[p, h // 2, i] for x, (p, i) in zip(w, rows)) / sum(w)
        assert np.allclose(r["out"][0, h], o)
        assert np.isclose(r["lse"][0, h], math.log(sum(w)))
    assert np.allclose(r["acc"][0, :, :7].sum(-1), 2.0) and np.isnan(r["acc"][0, :, 7:]).all()
    assert (r["out"][1] == 0).all() and (r["lse"][1] == -np.inf).all()


def test_attention_of_equal_scores_is_the_mean_and_a_mask_selects():
    k = np.zeros((2, 1, 4, 8))
    v = np.arange(8.0).reshape(2, 1, 4, 1) * np.ones(8)
    pages = np.array([[0, 1]], np.int32)
    q = np.ones((1, 1, 8))
    assert np.allclose(okv.attention(q, k, v, pages, [8], 1.0)["out"], 3.5)
    assert np.allclose(okv.attention(q, k, v, pages, [8], 1.0, window=2)["out"], 6.5)
    mask = np.full((1, 8), -np.inf)
    assert (okv.attention(q, k, v, pages, [8], 1.0, mask=mask)["out"] == 0).all()
    mask[0, 3] = -3.4e38
    assert np.allclose(okv.attention(q, k, v, pages, [8], 1.0, mask=mask)["out"], 3.0)


def test_evict_by_hand():
    k = np.arange(8.0).reshape(2, 1, 4, 1)
    pages = np.array([[1, 0]], np.int32)
    acc = np.array([[[5, 1, 3, 3, 9, 0, 3, 2]]], np.float32)
    pos = np.array([[[0, 1, 2, 3, 4, 5, 6, 7]]], np.int32)
    # position 7 is recent; of the others 9, 5 and the first 3 stay
    k2, v2, a2, p2, n2 = okv.evict(k, k + 10, pages, [8], [8], 4, 0, 1, acc, pos)
    assert n2.tolist() == [4]
    assert a2[0, 0, :4].tolist() == [5, 9, 3, 2] and p2[0, 0, :4].tolist() == [0, 4, 2, 7]
    assert k2[1, 0, :, 0].tolist() == [4, 0, 6, 3] and v2[1, 0, :, 0].tolist() == [14, 10, 16, 13]
    assert np.array_equal(k2[0], k[0])


def test_evict_ties_nan_and_held():
    k = np.zeros((1, 1, 6, 1))
    pages = np.zeros((1, 1), np.int32)
    acc = np.array([[[np.nan, 0.0, -0.0, 0.0, 7, 1]]], np.float32)
    pos = np.arange(6, dtype=np.int32).reshape(1, 1, 6)
    out = okv.evict(k, k, pages, [6], [6], 3, 1, 0, acc, pos)
    assert out[3][0, 0, :3].tolist() == [0, 4, 5]  # the sink (a NaN), 7 and 1
    out = okv.evict(k, k, pages, [6], [0], 3, 0, 0, acc, pos)  # all recent: the first stay
    assert out[3][0, 0, :3].tolist() == [0, 1, 2]
