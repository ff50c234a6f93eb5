"""GPU parity of wq_norm_rope, its gradient and wq_kv_append_norm against the f64 oracle.

Tolerances.  A head's sum of squares has at most 16 roundings in a lane and 5 in the shuffles, the
mean, the root and 1 / root one each, halved by the root: r is within 14 2^-24, and with the
products by r, w and the rotation's two and a sum a value is within 19 2^-24 < 2^-19 of the
magnitude of its terms (the mean's error, at most 22 2^-24 of mean |x|, is one of them); a 16-bit
output adds half a step.  The gradient has three such sums, each of them within 24 2^-24 of its
terms' magnitude beside the error of h: 2^-18 of the sum of those.  The sums over rows and heads
take up to 64 values one after another in a lane and 40 more: 128 2^-24 beside h's error."""
import numpy as np
import pytest
import torch

import gemv_transformer_gb300 as wq
from helpers import Guarded, dev, status_ok
from kv_helpers import Cache, bits, workspace
from oracle import tokens as ot
from tokens_helpers import HALF, KINDS, TORCH, angles

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def built():
    from gemv_transformer_gb300 import build
    build.build()
    wq.load()
    yield
    status_ok()


class Setting:
    """Weights, positions and a table of a case, on the host and as descriptors."""

    def __init__(self, g, n, d, rot, kind, pairs, flags=0, weight=True, bias=True, rows=300):
        self.kind, self.flags, self.pairs = kind, flags, pairs
        self.dealt, self.restart = bool(flags & ot.DEALT), bool(flags & ot.RESTART)
        self.inter = bool(flags & ot.INTERLEAVED)
        self.w = (1 + 0.3 * g.standard_normal(d)).astype(np.float32) if weight else None
        self.b = (0.2 * g.standard_normal(d)).astype(np.float32) if bias else None
        self.keep = [None if x is None else dev(x) for x in (self.w, self.b)]
        self.norm = wq.head_norm(kind, EPS, *self.keep)
        self.pos = g.integers(0, rows, (len(pairs), n)).astype(np.int32)
        self.pos[:, 0] = rows - 1
        self.table = angles(rows, max(rot // 2, 2))
        self.pos_dev, self.table_dev = dev(self.pos), dev(self.table)
        self.rope = wq.rope_axes(rot, flags, pairs, self.pos_dev, self.table_dev) if rot else None
        self.eps = float(np.float32(EPS))

    def cs(self):
        if not self.rope:
            return np.zeros((self.pos.shape[1], 0, 2))
        return ot.cos_sin(self.pairs, self.pos, self.table.astype(np.float64), self.dealt,
                          self.restart)

    def want(self, x):
        y, mag = ot.norm(x, self.kind, self.eps, self.w, self.b)
        return ot.turn(y, self.cs(), self.inter, mag=mag)


SHAPES = [  # n, heads, d, rot, pairs, flags
    (1, 1, 64, 64, [32], 0), (3, 5, 128, 128, [32, 16, 16], ot.DEALT),
    (17, 2, 96, 80, [20, 20], ot.RESTART | ot.INTERLEAVED), (5, 3, 80, 80, [20, 10, 10], 0),
    (4, 1, 7, 6, [3], 0), (2, 4, 256, 256, [50, 26, 26, 26], ot.DEALT | ot.RESTART),
    (1237, 3, 72, 36, [10, 8], ot.INTERLEAVED), (6, 7, 128, 64, [32], ot.INTERLEAVED),
    (9, 2, 16, 0, [0], 0), (2, 3, 250, 100, [30, 20], ot.DEALT), (700, 40, 128, 128, [64], 0),
    (3, 2, 64, 64, [0, 32, 0], 0), (5, 2, 8, 8, [2, 1, 1], 0)]


@pytest.mark.parametrize("n,h,d,rot,pairs,flags", SHAPES)
@pytest.mark.parametrize("kind", [ot.NONE, ot.RMS, ot.LAYER])
@pytest.mark.parametrize("otype,pad,shift", [("f32", 0, 0), ("bf16", 8, 8), ("f16", 3, 1)])
def test_norm_rope(n, h, d, rot, pairs, flags, kind, otype, pad, shift):
    g = np.random.default_rng(n * 1000 + d)
    s = Setting(g, n, d, rot, kind, pairs, flags, weight=kind != ot.RMS or n != 3, bias=n != 1)
    x = (3 * g.standard_normal((n, h, d)) + 0.5).astype(np.float32)
    stride = h * d + pad
    src = torch.full((n * stride + shift + 8,), 7.0, device="cuda")
    src[shift:shift + n * stride].view(n, stride)[:, :h * d] = dev(x.reshape(n, h * d))
    out = torch.full((n * stride + shift + 8,), 5.0, device="cuda", dtype=TORCH[otype])
    wq.check(wq.wq_norm_rope(n, h, d, s.norm, s.rope, src[shift:], stride, KINDS[otype],
                             out[shift:], stride))
    got = out.double().cpu().numpy()
    body = got[shift:shift + n * stride].reshape(n, stride)
    assert (got[:shift] == 5).all() and (got[shift + n * stride:] == 5).all()
    assert (body[:, h * d:] == 5).all()
    want, mag = s.want(x)
    tol = 2.0 ** -19 * mag + (HALF[otype] * np.abs(want) * (1 + 2.0 ** -10) if otype != "f32" else 0)
    if otype == "f16":
        tol = tol + 2.0 ** -25  # half a step of its subnormals
    assert (np.abs(body[:, :h * d].reshape(n, h, d) - want) <= tol).all()
    status_ok()


def test_in_place():
    g = np.random.default_rng(3)
    s = Setting(g, 9, 128, 128, ot.RMS, [32, 32])
    x = g.standard_normal((9, 4, 128)).astype(np.float32)
    buf = dev(x)
    wq.check(wq.wq_norm_rope(9, 4, 128, s.norm, s.rope, buf, 512, wq.WQ_F32, buf, 512))
    want, mag = s.want(x)
    assert (np.abs(buf.cpu().numpy() - want) <= 2.0 ** -19 * mag).all()


def test_equals_rope_without_norm():
    """One axis and no norm: wq_rope's bits."""
    g = np.random.default_rng(4)
    n, h, d, rot = 33, 6, 96, 64
    s = Setting(g, n, d, rot, ot.NONE, [rot // 2])
    x = dev(g.standard_normal((n, h * d)).astype(np.float32))
    a, b = torch.zeros_like(x), torch.zeros_like(x)
    wq.check(wq.wq_norm_rope(n, h, d, None, s.rope, x, h * d, wq.WQ_F32, a, h * d))
    wq.check(wq.wq_rope(n, h, d, rot, 0, x, h * d, s.pos_dev, s.table_dev, 300, b, h * d))
    assert torch.equal(a, b)


def test_bad_positions_leave_their_rows():
    g = np.random.default_rng(5)
    n, d = 6, 64
    s = Setting(g, n, d, d, ot.RMS, [16, 0, 16])
    s.pos[0, 1], s.pos[2, 3], s.pos[1, 4] = -1, 300, 1 << 30  # axis 1 turns nothing
    s.pos_dev.copy_(dev(s.pos))
    x = g.standard_normal((n, 2, d)).astype(np.float32)
    out = Guarded(n * 2 * d)
    before = out.view.clone()
    wq.check(wq.wq_norm_rope(n, 2, d, s.norm, s.rope, dev(x), 2 * d, wq.WQ_F32, out.view, 2 * d))
    assert wq.wq_get_device_status() == wq.WQ_ERR_BAD_INDEX
    got = out.result().reshape(n, 2, d)
    ok = [0, 2, 4, 5]
    s.pos = np.where((s.pos < 0) | (s.pos >= 300), 0, s.pos)
    want, mag = s.want(x)
    assert (np.abs(got[ok] - want[ok]) <= 2.0 ** -19 * mag[ok]).all()
    for t in (1, 3):
        assert np.isnan(got[t]).all()
        assert torch.equal(out.view.view(torch.int32).view(n, -1)[t],
                           before.view(torch.int32).view(n, -1)[t])


@pytest.mark.parametrize("kind", [ot.RMS, ot.LAYER])
def test_values_that_are_not_finite_stay_in_their_head(kind):
    g = np.random.default_rng(6)
    s = Setting(g, 4, 128, 128, kind, [64])
    x = g.standard_normal((4, 3, 128)).astype(np.float32)
    clean = x.copy()
    x[1, 1, 5], x[2, 0, 100] = np.nan, np.inf
    out = torch.zeros(4, 3, 128, device="cuda")
    wq.check(wq.wq_norm_rope(4, 3, 128, s.norm, s.rope, dev(x), 384, wq.WQ_F32, out, 384))
    got = out.cpu().numpy()
    want, mag = s.want(clean)
    for t in range(4):
        for h in range(3):
            if (t, h) in ((1, 1), (2, 0)):
                assert np.isnan(got[t, h]).any()
            else:
                assert (np.abs(got[t, h] - want[t, h]) <= 2.0 ** -19 * mag[t, h]).all()


def test_zero_heads():
    """A head of zeros: r = 1 / sqrt(eps), y = b; with eps 0 the formula has no value."""
    s = Setting(np.random.default_rng(1), 2, 64, 0, ot.RMS, [0])
    x = torch.zeros(2, 64, device="cuda")
    wq.check(wq.wq_norm_rope(2, 1, 64, s.norm, None, x, 64, wq.WQ_F32, x, 64))
    assert (x.cpu().numpy() == s.b).all()


def run_grad(s, x, g, aligned=True):
    n, h, d = x.shape
    size = wq.wq_norm_rope_grad_workspace_bytes(n, h, d)
    room = workspace(size)
    off = 0 if aligned else 1
    src, gr = (torch.zeros(n * h * d + 4, device="cuda")[off:off + n * h * d] for _ in range(2))
    src.copy_(dev(x.reshape(-1)))
    gr.copy_(dev(g.reshape(-1)))
    gx, gw, gb = Guarded(n * h * d), Guarded(d), Guarded(d)
    sums = s.kind != ot.NONE
    wq.check(wq.wq_norm_rope_grad(n, h, d, s.norm, s.rope, src, h * d, gr, h * d, gx.view, h * d,
                                  gw.view if sums else None, gb.view if sums else None, room,
                                  size))
    return (gx.result().reshape(n, h, d).astype(np.float64),
            *(v.result().astype(np.float64) if sums else None for v in (gw, gb)))


@pytest.mark.parametrize("n,h,d,rot,pairs,flags", SHAPES)
@pytest.mark.parametrize("kind", [ot.NONE, ot.RMS, ot.LAYER])
@pytest.mark.parametrize("aligned", [True, False])
def test_gradient(n, h, d, rot, pairs, flags, kind, aligned):
    g = np.random.default_rng(n * 1000 + d + 1)
    s = Setting(g, n, d, rot, kind, pairs, flags, weight=n != 3)
    x = (2 * g.standard_normal((n, h, d)) + 0.3).astype(np.float32)
    up = g.standard_normal((n, h, d)).astype(np.float32)
    got = run_grad(s, x, up, aligned)
    y, mag = ot.turn(up.astype(np.float64), s.cs(), s.inter, back=True)
    want = ot.norm_grad(x, y, kind, s.eps, s.w)
    if kind == ot.NONE:
        assert (np.abs(got[0] - want[0]) <= 2.0 ** -22 * mag).all()
        return
    hh, r = ot.hat(x, kind, s.eps)
    hmag = (np.abs(x) + np.abs(x).mean(-1, keepdims=True)) * r
    u = mag * (1 if s.w is None else np.abs(s.w))
    bound = r * (u + hmag * (u * hmag).mean(-1, keepdims=True) + u.mean(-1, keepdims=True))
    assert (np.abs(got[0] - want[0]) <= 2.0 ** -18 * bound).all()
    assert (np.abs(got[1] - want[1]) <= 2.0 ** -17 * (mag * hmag).sum((0, 1))).all()
    assert (np.abs(got[2] - want[2]) <= 2.0 ** -17 * mag.sum((0, 1))).all()
    status_ok()


@pytest.mark.parametrize("kind", [ot.RMS, ot.LAYER])
def test_gradient_against_differences(kind):
    """L = <up, f(x, w)>, its central difference along a random direction in f64 of the oracle's f,
    which the forward test ties to the library's: the step's own error is O(step^2)."""
    g = np.random.default_rng(11)
    n, h, d = 7, 2, 64
    s = Setting(g, n, d, d, kind, [16, 16], ot.DEALT)
    x = g.standard_normal((n, h, d)).astype(np.float32)
    up = g.standard_normal((n, h, d)).astype(np.float32)
    dx, dw, db = (g.standard_normal(v) for v in ((n, h, d), d, d))
    gx, gw, gb = run_grad(s, x, up)

    def value(e):
        y, _ = ot.norm(x + e * dx, kind, s.eps, s.w + e * dw, s.b + e * db)
        return (ot.turn(y, s.cs(), s.inter)[0] * up).sum()
    step = 1e-4
    diff = (value(step) - value(-step)) / (2 * step)
    grad = (gx * dx).sum() + (gw * dw).sum() + (gb * db).sum()
    size = (np.abs(gx * dx)).sum() + np.abs(gw * dw).sum() + np.abs(gb * db).sum()
    assert abs(diff - grad) <= 2.0 ** -16 * size + 100 * step ** 2 * size


def test_gradient_in_place_and_repeated_bits():
    g = np.random.default_rng(12)
    n, h, d = 300, 8, 128
    s = Setting(g, n, d, d, ot.LAYER, [64])
    x, up = (g.standard_normal((n, h, d)).astype(np.float32) for _ in range(2))
    first = run_grad(s, x, up)
    again = run_grad(s, x, up)
    assert all((a == b).all() for a, b in zip(first, again))
    size = wq.wq_norm_rope_grad_workspace_bytes(n, h, d)
    buf, room = dev(up), workspace(size)
    gw = torch.zeros(d, device="cuda")
    wq.check(wq.wq_norm_rope_grad(n, h, d, s.norm, s.rope, dev(x), h * d, buf, h * d, buf, h * d,
                                  gw, None, room, size))
    assert (buf.cpu().numpy() == first[0]).all() and (gw.cpu().numpy() == first[1]).all()


@pytest.mark.parametrize("kind,page,major,qtype", [("bf16", 16, "head", "bf16"),
                                                   ("f16", 7, "token", "f32"),
                                                   ("f32", 1, "gap", "f16"),
                                                   ("bf16", 64, "token", "f32")])
@pytest.mark.parametrize("hq,hkv,d,rot,pairs,flags", [
    (8, 2, 64, 64, [16, 8, 8], ot.DEALT), (5, 5, 128, 128, [64], 0), (0, 3, 80, 40, [20], 0),
    (6, 1, 256, 256, [64, 64], ot.INTERLEAVED), (3, 1, 24, 12, [4, 2], 0), (4, 2, 96, 0, [0], 0)])
@pytest.mark.parametrize("pad", [0, 3])
def test_append(kind, page, major, qtype, hq, hkv, d, rot, pairs, flags, pad):
    g = np.random.default_rng(d + page)
    lens = [5, 40, 0, 17]
    c = Cache(g, lens, hkv, d, kind, page, major, max_pages=-(-48 // page))
    # The last tokens of each sequence, one padding token among them.
    where = [(0, 4), (1, 38), (1, 39), (3, -1), (3, 16), (3, 0)]
    n = len(where)
    s = Setting(g, n, d, rot, ot.RMS, pairs, flags)
    k_norm = Setting(g, n, d, rot, ot.LAYER, pairs, flags)
    row = (hq + 2 * hkv) * d + pad
    x = (2 * g.standard_normal((n, row))).astype(np.float32)
    xd = dev(x)
    base = xd.data_ptr()
    q_out = torch.full((n, max(1, hq) * d + pad), 3.0, device="cuda", dtype=TORCH[qtype])
    slots = c.max_pages * page
    acc = torch.ones(4, hkv, slots, device="cuda")
    at = torch.full((4, hkv, slots), -7, device="cuda", dtype=torch.int32)
    before = c.host()
    seq, slot = (dev(np.array(v, np.int32)) for v in zip(*where))
    wq.check(wq.wq_kv_append_norm(
        c.desc, n, hq, s.norm, k_norm.norm, s.rope, base, row, base + 4 * hq * d, row,
        base + 4 * (hq + hkv) * d, row, 4, seq, slot, c.pages_dev, c.max_pages, KINDS[qtype],
        q_out, q_out.shape[1], acc, at if rot else None, slots))
    heads = x[:, :row - pad].reshape(n, hq + 2 * hkv, d)
    q_want, q_mag = s.want(heads[:, :hq])
    kn, km = ot.norm(heads[:, hq:hq + hkv], ot.LAYER, s.eps, k_norm.w, k_norm.b)
    k_want, k_mag = ot.turn(kn, s.cs(), s.inter, mag=km)
    sub = {"bf16": 0, "f16": 2.0 ** -25, "f32": 0}
    got_q = q_out.double().cpu().numpy()
    after = c.host()
    untouched = [np.ones(b.shape, bool) for b in before]
    for t, (i, j) in enumerate(where):
        if j < 0:
            assert (got_q[t] == 3).all()
            continue
        if hq:
            mine = got_q[t, :hq * d].reshape(hq, d)
            tol = 2.0 ** -19 * q_mag[t] + HALF[qtype] * 1.01 * np.abs(q_want[t]) + sub[qtype]
            assert (np.abs(mine - q_want[t]) <= tol).all() and (got_q[t, hq * d:] == 3).all()
        p, r = c.pages[i, j // page], j % page
        tol = 2.0 ** -19 * k_mag[t] + HALF[kind] * 1.01 * np.abs(k_want[t]) + sub[kind]
        assert (np.abs(after[0][p, :, r] - k_want[t]) <= tol).all()
        v = heads[t, hq + hkv:].astype(np.float64)
        assert (np.abs(after[1][p, :, r] - v) <= HALF[kind] * np.abs(v) + sub[kind]).all()
        for u in untouched:
            u[p, :, r] = False
        assert (acc[i, :, j] == 0).all()
        if rot:
            assert (at[i, :, j].cpu().numpy() == s.pos[0, t]).all()
    for b, a, u in zip(before, after, untouched):
        assert np.array_equal(b[u], a[u], equal_nan=True)
    assert int((acc == 0).sum()) == 5 * hkv
    status_ok()


def test_append_equals_kv_append():
    """Without norms and with one axis: wq_kv_append's bits."""
    g = np.random.default_rng(8)
    n, hq, hkv, d = 70, 4, 2, 64
    caches = [Cache(np.random.default_rng(1), [n], hkv, d) for _ in range(2)]
    s = Setting(g, n, d, d, ot.NONE, [d // 2])
    row = (hq + 2 * hkv) * d
    x = dev(g.standard_normal((n, row)).astype(np.float32))
    k, v = x[:, hq * d:], x[:, (hq + hkv) * d:]
    seq, slot = torch.zeros(n, dtype=torch.int32, device="cuda"), dev(np.arange(n, dtype=np.int32))
    outs = [torch.zeros(n, hq * d, device="cuda") for _ in range(2)]
    wq.check(wq.wq_kv_append_norm(caches[0].desc, n, hq, None, None, s.rope, x, row, k, row, v, row,
                                  1, seq, slot, caches[0].pages_dev, caches[0].max_pages,
                                  wq.WQ_F32, outs[0], hq * d))
    wq.check(wq.wq_kv_append(caches[1].desc, n, hq, d, 0, x, row, k, row, v, row, s.pos_dev,
                             s.table_dev, 300, 1, seq, slot, caches[1].pages_dev,
                             caches[1].max_pages, outs[1], hq * d))
    assert torch.equal(*outs)
    for a, b in zip(caches[0].pools, caches[1].pools):
        assert (bits(a) == bits(b)).all()


def test_append_refused_tokens_leave_everything():
    g = np.random.default_rng(9)
    c = Cache(g, [20, 20], 2, 64, max_pages=2)
    where = [(0, 3), (2, 1), (-1, 1), (1, 32), (1, 5), (0, 9)]
    n = len(where)
    s = Setting(g, n, 64, 64, ot.RMS, [32])
    s.pos_dev[0, 4] = 300
    c.pages_dev[0, 0] = 99  # slots 0..15 of sequence 0 have no page
    x = dev(g.standard_normal((n, 4 * 64)).astype(np.float32))
    out = torch.full((n, 128), 3.0, device="cuda")
    before = [bits(p) for p in c.pools]
    seq, slot = (dev(np.array(v, np.int32)) for v in zip(*where))
    k = torch.randn(n, 128, device="cuda")
    wq.check(wq.wq_kv_append_norm(c.desc, n, 2, s.norm, s.norm, s.rope, x, 256, k, 128, k, 128, 2,
                                  seq, slot, c.pages_dev, 2, wq.WQ_F32, out, 128))
    assert wq.wq_get_device_status() == wq.WQ_ERR_BAD_INDEX
    assert (out == 3).all()
    assert all((a == bits(p)).all() for a, p in zip(before, c.pools))


def test_captured_step_replays():
    """Forward, gradient and append in a graph, replayed on new values."""
    g = np.random.default_rng(10)
    n, h, d = 12, 4, 64
    s = Setting(g, n, d, d, ot.RMS, [32])
    x = dev(g.standard_normal((n, h * d)).astype(np.float32))
    y, gx, gw = torch.zeros_like(x), torch.zeros_like(x), torch.zeros(d, device="cuda")
    size = wq.wq_norm_rope_grad_workspace_bytes(n, h, d)
    room = workspace(size)

    def step():
        wq.check(wq.wq_norm_rope(n, h, d, s.norm, s.rope, x, h * d, wq.WQ_F32, y, h * d))
        wq.check(wq.wq_norm_rope_grad(n, h, d, s.norm, s.rope, x, h * d, y, h * d, gx, h * d, gw,
                                      None, room, size))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.copy_(torch.randn_like(x))
    graph.replay()
    torch.cuda.synchronize()
    got = [v.clone() for v in (y, gx, gw)]
    step()
    assert all(torch.equal(a, b) for a, b in zip(got, (y, gx, gw)))
