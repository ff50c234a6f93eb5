"""GPU parity of wq_rope_table and wq_rope against the f64 oracle.

Tolerances: a table value is one f32 rounding of an f64 value whose angle is off by at
most 2^-50 of up to 2^17: 2^-24 m.  A rotated value is two f32 products and a sum:
2^-24 (|a c| + |b s|) for the products and as much for the sum, so 2^-22 of them."""
import numpy as np
import pytest
import torch

import gemv_transformer_gb300 as wq
from helpers import Guarded, dev, status_ok
from oracle import kv as okv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from gemv_transformer_gb300 import build
    build.build()
    wq.load()
    yield
    status_ok()


def make_table(rows, rot, base=10000.0, scaling=None):
    out = Guarded(rows * rot)
    wq.check(wq.wq_rope_table(rows, rot, base, scaling, out.view), "wq_rope_table")
    return out


@pytest.mark.parametrize("rows,rot,base", [(1, 2, 10000.0), (7, 6, 10000.0), (513, 64, 500000.0),
                                           (131072, 128, 10000.0), (100, 256, 1.5)])
def test_table(rows, rot, base):
    got = make_table(rows, rot, base).result().reshape(rows, rot // 2, 2)
    assert (np.abs(got - okv.table(rows, rot, base)) <= 2.0 ** -24).all()


@pytest.mark.parametrize("kind", [wq.WQ_ROPE_LINEAR, wq.WQ_ROPE_NTK, wq.WQ_ROPE_YARN,
                                  wq.WQ_ROPE_BANDS])
@pytest.mark.parametrize("factor,magnitude", [(4.0, 0.0), (1.0, 1.25), (40.0, 0.0)])
def test_scaled_table(kind, factor, magnitude):
    rows, rot, base = 3000, 96, 10000.0
    sc = wq.RopeScaling(kind, 1024, factor, 1.0, 32.0, magnitude)
    got = make_table(rows, rot, base, sc).result().reshape(rows, rot // 2, 2)
    want = okv.table(rows, rot, base, magnitude or None, kind, factor, low=1.0, high=32.0,
                     original=1024)
    assert (np.abs(got - want) <= 2.0 ** -24 * np.abs(want).max()).all()


def run_rope(x, pos, table, rows, rot, flags, pad=0, shift=0, in_place=False):
    n, h, d = x.shape
    stride = h * d + pad
    buf = torch.full((n * stride + shift + 8,), 3.0, device="cuda")
    view = buf[shift:shift + n * stride].view(n, stride)
    view[:, :h * d] = dev(x.reshape(n, h * d))
    out = buf if in_place else torch.full_like(buf, 5.0)
    wq.check(wq.wq_rope(n, h, x.shape[2], rot, flags, buf[shift:], stride,
                        dev(np.asarray(pos, np.int32)), table, rows, out[shift:], stride),
             "wq_rope")
    torch.cuda.synchronize()
    host = out.cpu().numpy()
    rest = 3.0 if in_place else 5.0
    body = host[shift:shift + n * stride].reshape(n, stride)
    assert (host[:shift] == rest).all() and (host[shift + n * stride:] == rest).all()
    assert (body[:, h * d:] == rest).all()
    return body[:, :h * d].reshape(n, h, d)


@pytest.mark.parametrize("n,h,d,rot", [(1, 1, 64, 64), (3, 5, 128, 128), (17, 2, 96, 80),
                                       (2, 3, 80, 20), (4, 1, 7, 6), (1, 2, 6, 2),
                                       (33, 40, 128, 64), (5, 2, 256, 256), (3, 2, 9, 0),
                                       (1237, 3, 72, 36)])
@pytest.mark.parametrize("flags", [0, wq.WQ_ROPE_INTERLEAVED, wq.WQ_ROPE_TRANSPOSE,
                                   wq.WQ_ROPE_INTERLEAVED | wq.WQ_ROPE_TRANSPOSE])
@pytest.mark.parametrize("pad,shift,in_place", [(0, 0, False), (4, 4, True), (3, 1, False),
                                                (1, 2, True)])
def test_rope(n, h, d, rot, flags, pad, shift, in_place):
    g = np.random.default_rng(n * 1000 + d)
    x = g.standard_normal((n, h, d)).astype(np.float32)
    rows = 300
    pos = g.integers(0, rows, n)
    pos[0], pos[-1] = rows - 1, 0
    table = make_table(rows, rot).view if rot else None
    got = run_rope(x, pos, table, rows, rot, flags, pad, shift, in_place)
    cs = table.cpu().numpy().astype(np.float64).reshape(rows, rot // 2, 2)[pos] if rot else \
        np.zeros((n, 0, 2))
    want, mag = okv.rotate(x, cs, rot, flags)
    assert (np.abs(got - want) <= 2.0 ** -22 * mag).all()
    assert (got[..., rot:] == x[..., rot:]).all()
    status_ok()


def test_gradient_against_differences():
    """L(x) = <w, R x> is linear: its difference over a unit step is its gradient's product
    with the step; both sides are sums of n = 2880 terms in f64 of values within 2^-22."""
    g = np.random.default_rng(5)
    n, h, d, rot = 15, 2, 96, 64
    x, w, u = (g.standard_normal((n, h, d)).astype(np.float32) for _ in range(3))
    pos = g.integers(0, 500, n)
    table = make_table(500, rot).view
    for flags in (0, wq.WQ_ROPE_INTERLEAVED):
        lo, hi = (run_rope((x + e * u).astype(np.float32), pos, table, 500, rot, flags)
                  for e in (-1, 1))
        diff = ((hi.astype(np.float64) - lo) * w).sum() / 2
        grad = run_rope(w, pos, table, 500, rot, flags | wq.WQ_ROPE_TRANSPOSE).astype(np.float64)
        bound = 2.0 ** -22 * 4 * (np.abs(w) * (np.abs(x) + np.abs(u))).sum() * 2
        assert abs(diff - (grad * u).sum()) <= bound


def test_positions_out_of_range_leave_their_rows():
    g = np.random.default_rng(6)
    x = g.standard_normal((5, 2, 64)).astype(np.float32)
    table = make_table(10, 64).view
    pos = [3, -1, 10, 9, 1 << 30]
    got = run_rope(x, pos, table, 10, 64, 0)
    assert wq.wq_get_device_status() == wq.WQ_ERR_BAD_INDEX
    cs = table.cpu().numpy().astype(np.float64).reshape(10, 32, 2)
    for t in range(5):
        if 0 <= pos[t] < 10:
            want, mag = okv.rotate(x[t:t + 1], cs[[pos[t]]], 64)
            assert (np.abs(got[t:t + 1] - want) <= 2.0 ** -22 * mag).all()
        else:
            assert (got[t] == 5.0).all()


def test_infinities_and_nans_stay_in_their_pairs():
    x = np.ones((2, 1, 64), np.float32)
    x[0, 0, 3], x[1, 0, 40] = np.inf, np.nan
    got = run_rope(x, [5, 6], make_table(10, 64).view, 10, 64, 0)
    bad = ~np.isfinite(got)
    assert bad[0, 0].nonzero()[0].tolist() == [3, 35] and bad[1, 0].nonzero()[0].tolist() == [8, 40]


def test_long_rows_pass_32_bits():
    """Rows whose offsets pass 2^32 bytes: the last rows of a strided tensor."""
    n, stride, d = 33, 1 << 25, 64
    buf = torch.zeros(n * stride, device="cuda")
    x = torch.randn(n, d, generator=torch.Generator().manual_seed(1))
    buf.view(n, stride)[:, :d] = x.cuda()
    table = make_table(100, d).view
    pos = np.arange(n, dtype=np.int32)
    wq.check(wq.wq_rope(n, 1, d, d, 0, buf, stride, dev(pos), table, 100, buf, stride), "wq_rope")
    got = buf.view(n, stride)[:, :d].cpu().numpy()
    cs = table.cpu().numpy().astype(np.float64).reshape(100, d // 2, 2)[pos]
    want, mag = okv.rotate(x.numpy()[:, None], cs, d)
    assert (np.abs(got - want[:, 0]) <= 2.0 ** -22 * mag[:, 0]).all()
