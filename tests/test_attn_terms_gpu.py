"""wq_attn_paged where the operands' terms matter: values that are not finite, weights and
query components far below their largest, values with every mantissa bit set, large groups.

The bounds are the header's: a product within 2^-22 of exact, sums in f32.  They are derived
beside each test."""
import math

import numpy as np
import pytest
import torch

import gemv_transformer_gb300 as wq
from helpers import dev, status_ok
from kv_helpers import TYPES, Cache
from test_attn_paged_gpu import call, check, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from gemv_transformer_gb300 import build
    build.build()
    wq.load()
    yield
    status_ok()


def fill(c, k, v):
    """One sequence's slots as k, v [hkv][slots][d], given in f32."""
    for pool, x in zip(c.pools, (k, v)):
        x = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(TYPES[c.kind])
        for j in range(x.shape[1]):
            pool[c.pages[0, j // c.page], :, j % c.page] = x[:, j].cuda()


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("hq,d,lens", [(2, 64, [1, 40]), (8, 128, [1, 70]), (14, 64, [20, 3000]),
                                       (32, 128, [33, 5]), (6, 256, [1, 50]), (12, 128, [300, 90]),
                                       (20, 256, [7, 2500])])
def test_a_value_that_is_not_finite(kind, bad, hq, d, lens):
    """In k: every head that reads it; in v: its dim of them.  The query has components of either
    sign, some exact in any type, some with residuals of either sign, one 0."""
    g = np.random.default_rng(hq + d)
    near = np.array([1.0, 1 + 2.0 ** -12, 1 - 2.0 ** -13, -1 - 2.0 ** -12, -1 + 2.0 ** -9, 0.0, 3.0,
                     1 + 2.0 ** -20], np.float32)
    group = hq // 2
    for slot, dim in ((lens[1] - 1, 5), (0, d - 1)):
        for pool in (0, 1):
            c = Cache(g, lens, 2, d, kind, 16)
            q = queries(g, 2, hq, d)
            q[1, :, dim] = near[np.arange(hq) % len(near)]
            c.pools[pool][c.pages[1, slot // 16], 1, slot % 16, dim] = bad
            out, lse, _ = call(c, lens, hq, q, 0.125)
            assert np.isfinite(out[0]).all() and np.isfinite(lse[0]).all()
            assert np.isfinite(out[1, :group]).all() and np.isfinite(lse[1, :group]).all()
            mine = out[1, group:]
            if pool == 0:
                assert not np.isfinite(mine).any() and not np.isfinite(lse[1, group:]).any()
            else:
                assert not np.isfinite(mine[:, dim]).any() and np.isfinite(lse[1]).all()
                assert np.isfinite(np.delete(mine, dim, 1)).all()


def two_slots(kind, score, v, d=64, hq=2, extra=0):
    """Slots with scores 0 and `score` (from the mask; k is 0) and values v [2]."""
    c = Cache(np.random.default_rng(0), [2 + extra], 1, d, kind, 16)
    k, vals = np.zeros((1, 2 + extra, d), np.float32), np.zeros((1, 2 + extra, d), np.float32)
    vals[:, 0], vals[:, 1] = v[0], v[1]
    fill(c, k, vals)
    mask = np.full((1, 2 + extra), -np.inf, np.float32)
    mask[0, :2] = 0.0, score
    out, lse, _ = call(c, [2 + extra], hq, np.ones((1, hq, d), np.float32), 0.125, mask=mask)
    return out[0].astype(np.float64), c.host()[1][c.pages[0, 0], 0, :2, 0]


@pytest.mark.parametrize("kind", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("hq", [2, 5, 12])
@pytest.mark.parametrize("v", [(1e-7, 60000.0), (-6.1e-5, 50000.0), (1.0, 1.0), (0.0, 60000.0)])
def test_weights_far_below_the_largest(kind, hq, v):
    """Scores are exact here, so what is left is exp and the sums, 2^-19 of sum p |v|."""
    for score in (-3.0, -8.31, -12.5, -15.1, -19.4, -25.0, -30.2, -36.6, -50.3, -80.0):
        out, host = two_slots(kind, score, v, hq=hq)
        e = np.exp(np.float64(np.float32(score)))
        want = (host[0] + e * host[1]) / (1 + e)
        size = (abs(host[0]) + e * abs(host[1])) / (1 + e)
        assert (np.abs(out - want) <= 2.0 ** -19 * size).all(), (score, out[0, 0], want)


@pytest.mark.parametrize("kind", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("hq", [1, 7, 16])
def test_query_components_far_below_the_largest(kind, hq):
    """The largest component of each head meets a k of 0, a small one a k that is not: the score
    is one product, and with one slot lse is the score.  A product within 2^-22, and two roundings
    of 2^-24 where terms are added."""
    g = np.random.default_rng(hq)
    d, at = 64, 11
    for power in range(0, 81, 4):
        c = Cache(g, [1], 1, d, kind, 16)
        k, q = np.zeros((1, 1, d), np.float32), np.zeros((1, hq, d), np.float32)
        k[..., at] = 60000.0
        q[..., 3] = 1 + g.random(hq)
        q[..., at] = (1 + g.random(hq)) * 2.0 ** -power
        fill(c, k, k)
        _, lse, _ = call(c, [1], hq, q, 1.0)
        kk = c.host()[0][c.pages[0, 0], 0, 0, at]
        want = q[0, :, at].astype(np.float64) * kk
        assert (np.abs(lse[0] - want) <= (2.0 ** -22 + 2.0 ** -23) * np.abs(want)).all(), power


def test_spread_scores_and_values_of_every_size_f16():
    """Scores from 0 to -40 under values from 1e-7 to 6e4, the largest where the weights are
    least, whole rows and split ones.  The mask gives the scores, k is 0, so they are exact."""
    g = np.random.default_rng(3)
    d = 64
    for size, hq in ((64, 3), (900, 8), (9000, 2), (9000, 16)):
        c = Cache(g, [size], 1, d, "f16", 16)
        mask = -np.sort(40 * g.random(size)).astype(np.float32)[None]
        mask[0, 0] = 0.0
        v = (np.exp(-mask[0].astype(np.float64)) * 1e-7).clip(1e-7, 6e4)[:, None]
        v = v * g.choice([-1.0, 1.0], (size, d))
        order = g.permutation(size)
        mask, v = mask[:, order], v[order]
        fill(c, np.zeros((1, size, d)), v[None])
        out, lse, _ = call(c, [size], hq, np.ones((1, hq, d), np.float32), 0.125, mask=mask)
        vh = np.concatenate(list(c.host()[1][c.pages[0], 0]))[:size]
        p = np.exp(mask[0].astype(np.float64))
        p /= p.sum()
        assert (np.abs(out[0] - p @ vh) <= 2.0 ** -19 * (p @ np.abs(vh))).all()


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("hq", [3, 8, 16])
def test_small_values_beside_large_ones_of_no_weight(kind, hq):
    """In one tile: a v of 6e4 at a weight of e^-27, below f16's range, v of 6e-5 at weights near
    2^-10, v of 0 at the largest: sums may not be aligned to what is not there."""
    g = np.random.default_rng(hq)
    d = 64
    c = Cache(g, [16], 1, d, kind, 16)
    mask = (-10 * math.log(2) + 0.2 * g.standard_normal(16)).astype(np.float32)[None]
    mask[0, 0], mask[0, 9] = 0.0, -27.0
    v = 6e-5 * (1 + g.random((16, d)))
    v[0], v[9] = 0.0, 60000.0
    fill(c, np.zeros((1, 16, d)), v[None])
    out, _, _ = call(c, [16], hq, np.ones((1, hq, d), np.float32), 0.125, mask=mask)
    p = np.exp(mask[0].astype(np.float64))
    p /= p.sum()
    vh = c.host()[1][c.pages[0, 0], 0]
    assert (np.abs(out[0] - p @ vh) <= 2.0 ** -19 * (p @ np.abs(vh))).all()


# 24 significant bits whose low 13 are the most that two terms of 11 bits can lose.
FULL = 1 + 2.0 ** -11 + 2.0 ** -22 + 2.0 ** -23


def test_keys_and_values_of_24_bits_f32():
    """One slot: lse is the score, one product of q and k (scale 1, so q is not rounded before),
    within 2^-22 and two roundings of 2^-24 where terms are added; out is v times a weight of
    exactly 1, within 2^-22."""
    g = np.random.default_rng(4)
    d, hq = 64, 16
    for at in (0, 1, 2, 3, 17, 63):
        for size in (FULL, -FULL, 1000 * FULL, 2.0 ** -30 * FULL, 2 - 2.0 ** -23):
            c = Cache(g, [1], 2, d, "f32", 16)
            k = np.zeros((2, 1, d), np.float32)
            v = (size * (1 + 2.0 ** -23 * g.integers(0, 64, (2, 1, d)))).astype(np.float32)
            k[..., at] = size
            q = (1 + 2.0 ** -23 * g.integers(0, 1 << 23, (1, hq, d))).astype(np.float32)
            q[0, ::2, at] = (1 + 2.0 ** -23 * g.integers(0, 1 << 14, hq // 2)).astype(np.float32)
            fill(c, k, v)
            out, lse, _ = call(c, [1], hq, q, 1.0)
            want = q[0, :, at].astype(np.float64) * np.float64(np.float32(size))
            assert (np.abs(lse[0] - want) <= (2.0 ** -22 + 2.0 ** -23) * np.abs(want)).all(), (at, size)
            v = np.repeat(v[:, 0], hq // 2, 0).astype(np.float64)
            assert (np.abs(out[0] - v) <= 2.0 ** -22 * np.abs(v)).all(), size


@pytest.mark.parametrize("n,length,hq,hkv", [(1, 700, 12000, 1), (1, 3000, 9600, 1),
                                             (2, 40, 20100, 2)])
def test_weights_of_a_group_of_thousands(n, length, hq, hkv):
    g = np.random.default_rng(hq)
    lens = [length - 3 * i for i in range(n)]
    c = Cache(g, lens, hkv, 8, "bf16", 16)
    acc_in = np.abs(g.standard_normal((n, hkv, c.max_pages * 16))).astype(np.float32)
    check(c, lens, hq, queries(g, n, hq, 8), 0.35, acc_in=acc_in, with_acc=True)
