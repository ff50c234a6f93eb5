"""Queries and keys of wq_attn_tokens at the ends of their range, against the f64 oracle (its formulas
hold for infinities too).  Tolerances are those of test_attn_tokens_gpu; a capped score of an infinite
query is the cap itself, within 8 units of the last place and the tanh's 2^-21 of the cap."""
import numpy as np
import pytest
import torch

import gemv_transformer_gb300 as wq
from helpers import status_ok
from test_attn_tokens_gpu import TYPES, U, Case

pytestmark = pytest.mark.gpu
CACHES = ["bf16", "f16", "f32"]


@pytest.fixture(scope="module", autouse=True)
def built():
    from gemv_transformer_gb300 import build
    build.build()
    wq.load()
    yield
    status_ok()


@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("tree", [False, True])
def test_infinite_queries_under_a_cap(kind, d, tree):
    """Some heads' queries have an infinity: their scores are the cap with k's sign."""
    cap = 3.0
    c = Case(30, [20, 70], [40, 100], 4, 2, d, kind, "f32", tree=tree, softcap=cap)
    for t in (3, 25, 80):
        for h, value in ((0, np.inf), (2, -np.inf)):
            c.q[t, h * d + 9] = value
            c.q64[t, h * d + 9] = value
    c.run()
    w = c.want()
    sx = np.where(np.isinf(w["sx"]), cap, w["sx"])
    assert np.isinf(w["sx"]).sum() == 6 and np.isfinite(w["out"]).all()
    ex = (d + 8) * U * sx + 8 * U * w["mx"] + 2.0 ** -21 * cap
    n = w["n"][:, None]
    tol = (2 * ex + (n + 80) * U)[..., None] * w["pv"]
    got = c.out.double().cpu().numpy().reshape(c.m, 4, d)
    assert (np.abs(got - w["out"]) <= tol).all()
    lse = c.lse.double().cpu().numpy()
    none = np.isneginf(w["lse"])
    assert (np.isneginf(lse) == none).all()
    with np.errstate(invalid="ignore"):
        assert (none | (np.abs(lse - w["lse"]) <= ex + (n + 16) * U + 4 * U * np.abs(w["lse"]))).all()


@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("value", [3.4e38, -3.4028e38, 3.3895e38])
def test_queries_beyond_the_largest_bf16(kind, value):
    """Finite queries that bf16 rounds to infinity, with scores of a few units."""
    c = Case(31, [20, 70], [40, 100], 4, 2, 64, kind, "f32", scale=1e-37, qscale=1e36)
    for pool in c.cache.pools:
        pool[..., 9] *= 0.125
    for t in (0, 3, 25, 80):
        for h in range(4):
            c.q[t, h * 64 + 9] = value
            c.q64[t, h * 64 + 9] = float(np.float32(value))
    c.run().check()


@pytest.mark.parametrize("kind", CACHES)
def test_infinite_queries_without_a_cap(kind):
    """Their heads' results are not numbers, the others are as they were."""
    c = Case(32, [20, 70], [40, 100], 4, 2, 64, kind, "f32").run()
    before = c.out.clone()
    bad = np.zeros((c.m, 4), bool)
    for t, h, value in ((3, 0, np.inf), (25, 3, -np.inf), (80, 1, np.nan)):
        c.q[t, h * 64 + 9] = value
        bad[t, h] = True
    c.run()
    got, was = (x.cpu().numpy().reshape(c.m, 4, 64) for x in (c.out, before))
    assert (got[~bad] == was[~bad]).all() and np.isnan(got[bad]).all()


@pytest.mark.parametrize("kind,qtype", TYPES)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("value", [np.inf, -np.inf])
def test_infinite_keys(kind, qtype, d, value):
    """A token that sees one has a score of plus infinity, and NaN, or of minus infinity, and a weight
    of 0; f32 queries over bf16 may have NaN there too.  The others' results are without it."""
    c = Case(33, [20, 70], [40, 100], 4, 2, d, kind, qtype)
    w0 = c.want()
    s, j = 1, 100 + 30
    c.cache.pools[0][int(c.cache.pages[s, j // 16]), :, j % 16, 7] = value
    c.run()
    with np.errstate(all="ignore"):
        w = c.want()
    sees = np.zeros((c.m, 4), bool)
    sees[20 + 30:] = True
    up = sees & np.isnan(w["lse"])
    assert up.any() and (sees & ~up).any() and (up == np.isnan(w["out"]).all(-1)).all()
    got = c.out.double().cpu().numpy().reshape(c.m, 4, d)
    assert np.isnan(got[up]).all() and np.isnan(c.lse.cpu().numpy()[up]).all()
    void = up
    if (kind, qtype) == ("bf16", "f32"):
        void = sees & np.isnan(got).all(-1)
        assert (np.isnan(c.lse.cpu().numpy()) == void).all()
    # Compare what is left: scores' sizes are those without the infinity.
    for name in ("out", "lse", "pv"):
        w[name][void] = 0
    w["sx"], w["mx"] = w0["sx"], w0["mx"]
    c.out.view(c.m, 4, d)[torch.from_numpy(void).cuda()] = 0
    c.lse[torch.from_numpy(void).cuda()] = 0
    c.check(w)


@pytest.mark.parametrize("kind,qtype", TYPES)
def test_the_largest_and_the_least_cap(kind, qtype):
    """A cap of 2^60 changes no score by more than its roundings (8 units of the last place of the
    score), one of 2^-60 makes all weights alike."""
    c = Case(34, [20, 70], [40, 100], 4, 2, 128, kind, qtype, softcap=2.0 ** 60).run()
    c.softcap = 0.0
    c.check()
    Case(35, [20, 70], [40, 100], 4, 2, 64, kind, qtype, softcap=2.0 ** -60).run().check()
