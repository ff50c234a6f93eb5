"""The gradient of head norms where rows have positions out of range: those rows of grad_x stay as they
were and add nothing to the sums.  Tolerances as in test_norm_rope_gpu."""
import numpy as np
import pytest
import torch

import gemv_transformer_gb300 as wq
from helpers import Guarded, status_ok
from oracle import tokens as ot
from test_norm_rope_gpu import Setting, dev, run_grad

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from gemv_transformer_gb300 import build
    build.build()
    wq.load()
    yield
    status_ok()


@pytest.mark.parametrize("pairs,flags", [([32], 0), ([32], ot.INTERLEAVED), ([16, 0, 16], 0),
                                         ([16, 16], ot.DEALT | ot.RESTART)])
@pytest.mark.parametrize("kind", [ot.NONE, ot.RMS, ot.LAYER])
@pytest.mark.parametrize("h", [1, 5])
@pytest.mark.parametrize("n", [6, 900])
@pytest.mark.parametrize("aligned", [True, False])
def test_bad_positions(pairs, flags, kind, h, n, aligned):
    g = np.random.default_rng(n + h)
    d = 64
    s = Setting(g, n, d, d, kind, pairs, flags)
    bad = sorted({1, 3, n - 1, n // 2})
    for i, t in enumerate(bad):
        s.pos[-1 if i % 2 else 0, t] = (-1, 300, 1 << 30, -(1 << 31))[i % 4]
    if len(pairs) == 3:
        s.pos[1, 0] = 1 << 30  # that axis turns nothing
    s.pos_dev.copy_(dev(s.pos))
    x = (2 * g.standard_normal((n, h, d)) + 0.3).astype(np.float32)
    up = g.standard_normal((n, h, d)).astype(np.float32)
    gx, gw, gb = run_grad(s, x, up, aligned)
    assert wq.wq_get_device_status() == wq.WQ_ERR_BAD_INDEX
    ok = np.setdiff1d(np.arange(n), bad)
    assert np.isnan(gx[bad]).all() and np.isfinite(gx[ok]).all()  # the guards' pattern is a NaN
    s.pos[(s.pos < 0) | (s.pos >= 300)] = 0
    y, mag = ot.turn(up.astype(np.float64), s.cs(), s.inter, back=True)
    x, y, mag = x[ok], y[ok], mag[ok]
    want = ot.norm_grad(x, y, kind, s.eps, s.w)
    if kind == ot.NONE:
        assert (np.abs(gx[ok] - want[0]) <= 2.0 ** -22 * mag).all()
        return
    _, r = ot.hat(x, kind, s.eps)
    hmag = (np.abs(x) + np.abs(x).mean(-1, keepdims=True)) * r
    u = mag * np.abs(s.w)
    bound = r * (u + hmag * (u * hmag).mean(-1, keepdims=True) + u.mean(-1, keepdims=True))
    assert (np.abs(gx[ok] - want[0]) <= 2.0 ** -18 * bound).all()
    assert (np.abs(gw - want[1]) <= 2.0 ** -17 * (mag * hmag).sum((0, 1))).all()
    assert (np.abs(gb - want[2]) <= 2.0 ** -17 * mag.sum((0, 1))).all()


def test_no_row_is_in_range():
    """Sums of nothing are 0."""
    g = np.random.default_rng(1)
    s = Setting(g, 5, 64, 64, ot.RMS, [32])
    s.pos_dev.fill_(300)
    x = g.standard_normal((5, 2, 64)).astype(np.float32)
    gx, gw, gb = run_grad(s, x, x)
    assert wq.wq_get_device_status() == wq.WQ_ERR_BAD_INDEX
    assert np.isnan(gx).all() and (gw == 0).all() and (gb == 0).all()


def test_in_place_rows_out_of_range_keep_what_they_hold():
    g = np.random.default_rng(2)
    s = Setting(g, 9, 64, 64, ot.LAYER, [32])
    s.pos[0, [2, 7]] = 300, -5
    s.pos_dev.copy_(dev(s.pos))
    x, up = (g.standard_normal((9, 3 * 64)).astype(np.float32) for _ in range(2))
    buf = Guarded(9 * 192, up)
    wq.check(wq.wq_norm_rope_grad(9, 3, 64, s.norm, s.rope, dev(x), 192, buf.view, 192, buf.view,
                                  192))
    assert wq.wq_get_device_status() == wq.WQ_ERR_BAD_INDEX
    got = buf.result().reshape(9, 192)
    assert (got[[2, 7]] == up[[2, 7]]).all() and (got[[0, 1, 8]] != up[[0, 1, 8]]).any()
    torch.cuda.synchronize()
