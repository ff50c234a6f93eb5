"""wq_attn_tokens with more row tiles than its plan holds on the chip (2048), and more than it sums at a
time (1024), against the f64 oracle."""
import numpy as np
import pytest

import gemv_transformer_gb300 as wq
from helpers import status_ok
from test_attn_tokens_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from gemv_transformer_gb300 import build
    build.build()
    wq.load()
    yield
    status_ok()


@pytest.mark.parametrize("kind,qtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("heads", [(1, 1), (2, 2)])
def test_thousands_of_short_sequences(kind, qtype, heads):
    g = np.random.default_rng(40)
    counts = [int(x) for x in g.integers(1, 3, 2600)]
    contexts = [int(x) for x in g.integers(0, 21, 2600)]
    Case(40, counts, contexts, *heads, 64, kind, qtype, page=8).run().check()


@pytest.mark.parametrize("kind,qtype", [("bf16", "bf16"), ("f32", "f32")])
def test_long_ones_among_and_behind_them(kind, qtype):
    """Row tiles of many key tiles on both sides of the 2048th, cut by ranges of CTAs."""
    g = np.random.default_rng(41)
    counts = [int(x) for x in g.integers(1, 3, 2300)]
    contexts = [int(x) for x in g.integers(0, 9, 2300)]
    for s, (count, context) in {1000: (3, 2000), 2046: (150, 900), 2047: (9, 3000), 2048: (140, 700),
                                2299: (40, 2500)}.items():
        counts[s], contexts[s] = count, context
    Case(41, counts, contexts, 2, 1, 64, kind, qtype, page=8).run().check()


def test_many_row_tiles_of_one_sequence():
    """8200 tokens of 40 heads to a kv head: 2563 row tiles of 128, whose tokens see 30 slots each."""
    c = Case(42, [8200], [5], 40, 1, 8, "bf16", "f32", page=64, window=30)
    c.run()
    # The oracle for the tokens around the borders of the plan's parts.
    import torch
    from oracle import tokens as ot
    hk, hv = c.cache.host()
    got, lse = c.out.double().cpu().numpy(), c.lse.double().cpu().numpy()
    assert torch.isfinite(c.out).all() and torch.isfinite(c.lse).all()
    for j in (0, 1, 29, 30, 3276, 3277, 6552, 6553, 6554, 6555, 8198, 8199):
        q = c.q64[j, :320].reshape(1, 40, 8)
        # One new token behind j + 5 slots is the same row.
        w = ot.attention(q, hk, hv, c.cache.pages, [0, 1], [5 + j + 1], c.scale, window=30)
        u = 2.0 ** -24
        ex = (8 + 8) * u * w["sx"] + 8 * u * w["mx"]
        tol = (2 * ex + (30 + 80) * u)[..., None] * w["pv"]
        assert (np.abs(got[j, :320].reshape(1, 40, 8) - w["out"]) <= tol).all(), j
        assert (np.abs(lse[j] - w["lse"]) <= ex + 46 * u + 4 * u * np.abs(w["lse"])).all(), j
