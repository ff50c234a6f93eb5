"""wq_attn_paged where the operands' terms matter: values that are not finite, weights and
query components far below their largest, values with every mantissa bit set, large groups.

The bounds are the header's: a product within 2^-22 of exact, sums in f32, and for f16 caches a
floor (below).  They are derived beside each test."""
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
                                       (32, 128, [33, 5]), (6, 256, [1, 50])])
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
