"""GPU parity of wq_attn_paged against the f64 oracle.

Tolerances.  A score is a dot product of at most 256 exact-to-2^-22 products summed in f32:
its error is within e = 2^-19 scale sum|q k| + 2^-22 max|x| (a chain of 256 roundings of 2^-24
that add up as their square root, four times over, and the final scale and mask).  With
scores off by e the weights are off by a factor 1 +- 2e; exp, the sums of the weights and of
the products add 2^-19 in the same way.  So out is within (2e + 2^-19) sum p|v|, lse
within e + 2^-20 (1 + |lse|), a slot's weight within (2e + 2^-19) p + 2^-22 |acc_in|."""
import numpy as np
import pytest
import torch

import gemv_transformer_gb300 as wq
from helpers import dev, status_ok
from kv_helpers import Cache, bits, workspace
from oracle import kv as okv

pytestmark = pytest.mark.gpu
CAN = 12345.0


@pytest.fixture(scope="module", autouse=True)
def built():
    from gemv_transformer_gb300 import build
    build.build()
    wq.load()
    yield
    status_ok()


def call(c, lens, hq, q, scale, window=0, mask=None, acc_in=None, with_acc=False, in_place=False,
         pad=0, stride=None, stream=None):
    """The device's (out, lse, acc or None), with guards around each."""
    n, d = len(lens), c.d
    row = hq * d + pad
    qd = torch.full((n, row), float("nan"), device="cuda")
    qd[:, :hq * d] = dev(q.reshape(n, -1))
    out = torch.full((n + 1, row), CAN, device="cuda")
    lse = torch.full((n * hq + 1,), CAN, device="cuda")
    stride = stride or c.max_pages * c.page
    acc = ain = None
    if with_acc:
        acc = torch.full((n * c.hkv * stride + 1,), CAN, device="cuda")
        if acc_in is not None:
            ain = torch.full_like(acc, CAN)
            ain[:-1].view(n, c.hkv, stride)[:, :, :acc_in.shape[2]] = dev(acc_in)
            if in_place:
                acc = ain
    maskd = dev(mask) if mask is not None else None
    size = wq.wq_attn_paged_workspace_bytes(c.desc, n, hq, c.max_pages, with_acc)
    room = workspace(size)
    lensd = dev(np.asarray(lens, np.int32))
    torch.cuda.synchronize()
    wq.check(wq.wq_attn_paged(c.desc, n, hq, scale, window, qd, row, c.pages_dev, c.max_pages,
                              lensd, maskd, 0 if mask is None else mask.shape[1], out, row, lse,
                              ain, acc, stride, room, size, stream=stream), "wq_attn_paged")
    torch.cuda.synchronize()
    assert (out[n] == CAN).all() and (out[:n, hq * d:] == CAN).all() and lse[-1] == CAN
    if with_acc:
        assert acc[-1] == CAN
        acc = acc[:-1].view(n, c.hkv, stride).cpu().numpy()
    return (out[:n, :hq * d].cpu().numpy().reshape(n, hq, d), lse[:-1].cpu().numpy().reshape(n, hq),
            acc)


def check(c, lens, hq, q, scale, window=0, mask=None, acc_in=None, with_acc=False, want=None, **kw):
    out, lse, acc = call(c, lens, hq, q, scale, window, mask, acc_in, with_acc, **kw)
    k, v = c.host()
    r = want or okv.attention(q, k, v, c.pages, lens, scale, window, mask, acc_in)
    e = 2.0 ** -19 * r["sx"] + 2.0 ** -22 * r["mx"]
    assert (np.abs(out - r["out"]) <= (2 * e + 2.0 ** -19)[..., None] * r["pv"] + 1e-37).all(), \
        np.abs(out - r["out"]).max()
    none = r["lse"] == -np.inf
    assert (lse[none] == -np.inf).all() and (out[none] == 0).all()
    far = np.abs(lse[~none] - r["lse"][~none])
    assert (far <= e[~none] + 2.0 ** -20 * (1 + np.abs(r["lse"][~none]))).all()
    if with_acc:
        eg = e.reshape(len(lens), c.hkv, -1).max(-1)[..., None]
        slots = c.max_pages * c.page
        live = ~np.isnan(r["acc"])
        got, want_acc = acc[:, :, :slots], r["acc"]
        base = np.abs(acc_in[:, :, :slots]) if acc_in is not None else 0 * want_acc
        tol = (2 * eg + 2.0 ** -19) * r["p"] + 2.0 ** -22 * base + 1e-37
        assert (np.abs(got - want_acc)[live] <= tol[live]).all()
        if not kw.get("in_place"):
            assert (got[~live] == CAN).all() and (acc[:, :, slots:] == CAN).all()
    status_ok()
    return out, lse, acc


def queries(g, n, hq, d, scale=1.0):
    return (scale * g.standard_normal((n, hq, d))).astype(np.float32)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 64), (8, 1, 128), (6, 2, 96), (3, 3, 80), (9, 1, 64),
                                      (16, 1, 128), (24, 1, 256), (20, 4, 192), (2, 1, 8),
                                      (35, 1, 72), (64, 2, 136)])
def test_heads_and_types(kind, hq, hkv, d):
    g = np.random.default_rng(hq * 1000 + d)
    lens = [0, 1, 15, 16, 17, 63, 64, 65, 130]
    c = Cache(g, lens, hkv, d, kind, 16)
    check(c, lens, hq, queries(g, len(lens), hq, d), d ** -0.5)


@pytest.mark.parametrize("page", [1, 7, 16, 33, 64, 100, 256])
@pytest.mark.parametrize("major", ["head", "token", "gap"])
def test_pages_and_layouts(page, major):
    g = np.random.default_rng(page)
    lens = [200, 1, 64, 129, 300, 7]
    c = Cache(g, lens, 2, 64, "bf16", page, major, max_pages=-(-301 // page) + 2)
    acc_in = np.abs(g.standard_normal((6, 2, c.max_pages * page))).astype(np.float32)
    check(c, lens, 8, queries(g, 6, 8, 64), 0.125, acc_in=acc_in, with_acc=True, pad=4)


@pytest.mark.parametrize("n,length,hq,hkv,d,kind", [
    (1, 20011, 8, 2, 128, "bf16"), (1, 9000, 4, 4, 64, "f16"), (2, 7777, 12, 1, 256, "f32"),
    (1, 70001, 2, 1, 64, "bf16"), (3, 4099, 40, 8, 128, "bf16")])
@pytest.mark.parametrize("with_acc", [False, True])
def test_long(n, length, hq, hkv, d, kind, with_acc):
    g = np.random.default_rng(length)
    lens = [length - 1000 * i for i in range(n)]
    c = Cache(g, lens, hkv, d, kind, 64)
    check(c, lens, hq, queries(g, n, hq, d), d ** -0.5, with_acc=with_acc)


@pytest.mark.parametrize("seed", range(3))
def test_ragged_batch(seed):
    """Many sequences whose lengths have nothing in common, empty ones among them."""
    g = np.random.default_rng(100 + seed)
    n = [150, 37, 300][seed]
    lens = [int(x) for x in np.where(g.random(n) < 0.1, 0, g.integers(1, 700, n))]
    c = Cache(g, lens, 2, 64, "bf16", 16)
    acc_in = np.abs(g.standard_normal((n, 2, c.max_pages * 16))).astype(np.float32)
    check(c, lens, 4, queries(g, n, 4, 64), 0.125, window=[0, 100, 1][seed], acc_in=acc_in,
          with_acc=True, in_place=seed == 1)


@pytest.mark.parametrize("window", [1, 5, 16, 64, 100, 1000])
def test_windows(window):
    g = np.random.default_rng(window)
    lens = [0, 1, 99, 100, 101, 500, 1777]
    c = Cache(g, lens, 2, 128, "bf16", 16)
    k, v = (p for p in c.pools)
    for s, size in enumerate(lens):  # what lies before the window is not read
        for j in range(max(0, size - window)):
            k[c.pages[s, j // 16], :, j % 16] = float("nan")
            v[c.pages[s, j // 16], :, j % 16] = float("inf")
    check(c, lens, 8, queries(g, 7, 8, 128), 0.1, window=window, with_acc=True)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
def test_masks(kind):
    """A bias, -inf in places that hold NaN and infinities, the lowest value, nothing left."""
    g = np.random.default_rng(7)
    lens = [300, 300, 300, 90, 33, 300]
    c = Cache(g, lens, 2, 64, kind, 16)
    low = np.finfo(np.float32).min
    mask = (3 * g.standard_normal((6, 307))).astype(np.float32)
    mask[0, ::3] = -np.inf
    mask[1, :] = -np.inf
    mask[2, :] = low                    # all alike: the mean of the values
    mask[3, 40:] = low
    mask[4, :32] = -np.inf
    mask[5, 17:290] = -np.inf
    mask[:, 300:] = np.nan              # beyond the lengths
    for s, size in enumerate(lens):
        for j in range(size):
            if mask[s, j] == -np.inf:
                bad = [float("nan"), float("inf"), -float("inf")][j % 3]
                c.pools[0][c.pages[s, j // 16], :, j % 16] = bad
                c.pools[1][c.pages[s, j // 16], :, (j % 16)] = bad
    acc_in = np.abs(g.standard_normal((6, 2, c.max_pages * 16))).astype(np.float32)
    out, _, _ = check(c, lens, 6, queries(g, 6, 6, 64), 0.125, mask=mask, acc_in=acc_in,
                      with_acc=True)
    assert np.isfinite(out).all()


def test_large_scores_and_one_hot_weights():
    g = np.random.default_rng(8)
    lens = [500, 64, 1]
    c = Cache(g, lens, 1, 128, "f32", 16, scale=30.0)
    check(c, lens, 4, queries(g, 3, 4, 128, 30.0), 1.0, with_acc=True)
    check(c, lens, 4, queries(g, 3, 4, 128, 30.0), -1.0)
    check(c, lens, 4, queries(g, 3, 4, 128, 1e-30), 1.0)


def test_large_and_small_magnitudes():
    """f16 values at the ends of their range, queries far from one."""
    g = np.random.default_rng(9)
    lens = [200, 31]
    for kind, ks, qs in (("f16", 10000.0, 1e-4), ("f16", 1e-6, 1e5), ("bf16", 1e30, 1e-30),
                         ("f32", 1e-30, 1e30), ("bf16", 1e-30, 1e30)):
        c = Cache(g, lens, 2, 64, kind, 16, scale=ks)
        check(c, lens, 4, queries(g, 2, 4, 64, qs), 0.125)


def test_a_nan_that_takes_part_reaches_its_head_alone():
    g = np.random.default_rng(10)
    lens = [100, 100]
    c = Cache(g, lens, 2, 64, "bf16", 16)
    c.pools[0][c.pages[0, 3], 1, 2, 5] = float("nan")
    out, lse, _ = call(c, lens, 4, queries(g, 2, 4, 64), 0.125)
    assert np.isnan(out[0, 2:]).all() and np.isnan(lse[0, 2:]).all()
    assert np.isfinite(out[0, :2]).all() and np.isfinite(out[1]).all()


def test_same_bits_every_time_and_on_another_stream():
    g = np.random.default_rng(11)
    lens = [3000, 17, 801, 5000]
    c = Cache(g, lens, 2, 128, "bf16", 16)
    q = queries(g, 4, 16, 128)
    first = call(c, lens, 16, q, 0.1, with_acc=True)
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream):
        again = call(c, lens, 16, q, 0.1, with_acc=True, stream=stream)
        for a, b in zip(first, again):
            assert np.array_equal(a, b)


def test_a_sequence_gives_the_same_alone_as_in_a_batch_within_tolerance():
    g = np.random.default_rng(12)
    lens = [700, 64, 1500]
    c = Cache(g, lens, 2, 64, "bf16", 16)
    q = queries(g, 3, 4, 64)
    check(c, lens, 4, q, 0.125)
    whole = c.pages_dev
    for s in range(3):
        c.pages_dev = whole[s:s + 1].contiguous()
        pages, c.pages = c.pages, c.pages[s:s + 1]
        check(c, lens[s:s + 1], 4, q[s:s + 1], 0.125)
        c.pages = pages


def test_lengths_and_pages_out_of_range():
    g = np.random.default_rng(13)
    lens = [96, 96, -5]
    c = Cache(g, lens, 1, 64, "bf16", 16)
    q = queries(g, 3, 2, 64)
    k, v = c.host()
    # longer than the table: cut
    out, lse, _ = call(c, [1000, 96, -5], 2, q, 0.125)
    assert wq.wq_get_device_status() == wq.WQ_ERR_BAD_INDEX
    r = okv.attention(q, k, v, c.pages, lens, 0.125)
    assert np.allclose(out, r["out"], atol=1e-4) and (out[2] == 0).all()
    # pages that are not there: left out
    c.pages[0, 2], c.pages[1, :] = -1, 10 ** 6
    c.pages_dev = dev(c.pages)
    acc_in = np.ones((3, 1, 96), np.float32)
    out, lse, acc = call(c, lens, 2, q, 0.125, acc_in=acc_in, with_acc=True)
    assert wq.wq_get_device_status() == wq.WQ_ERR_BAD_INDEX
    r = okv.attention(q, k, v, c.pages, lens, 0.125, acc_in=acc_in)
    assert np.allclose(out, r["out"], atol=1e-4)
    assert (out[1:] == 0).all() and (lse[1:] == -np.inf).all()
    assert (acc[0, 0, 32:48] == 1).all() and (acc[1] == 1).all()
    assert np.allclose(acc[0], r["acc"][0], atol=1e-4)


def test_strides_of_sums_and_masks_cut_the_length():
    g = np.random.default_rng(14)
    c = Cache(g, [96, 50], 1, 64, "bf16", 16)
    q = queries(g, 2, 2, 64)
    acc_in = np.ones((2, 1, 61), np.float32)
    out, _, acc = call(c, [96, 50], 2, q, 0.125, acc_in=acc_in, with_acc=True, stride=61)
    assert wq.wq_get_device_status() == wq.WQ_ERR_BAD_INDEX
    k, v = c.host()
    r = okv.attention(q, k, v, c.pages, [61, 50], 0.125)
    assert np.allclose(out, r["out"], atol=1e-4)


@pytest.mark.parametrize("with_acc", [False, True])
def test_cache_beyond_4_gib(with_acc):
    """Slots whose byte offsets pass 2^32, in pages far apart."""
    g = np.random.default_rng(15)
    pages, page, d, step = 5, 16, 64, (1 << 30) + 64
    room = torch.empty(pages * step, dtype=torch.bfloat16, device="cuda")
    lens = [75]
    c = Cache(g, lens, 1, d, "bf16", page)
    k = room.as_strided((pages, 1, page, d), (step, page * d, d, 1))
    v = room[4096:].as_strided((pages, 1, page, d), (step, page * d, d, 1))
    order = [4, 0, 3, 1, 2]
    for i, p in enumerate(order):
        k[p], v[p] = c.pools[0][c.pages[0, i]], c.pools[1][c.pages[0, i]]
    c.pools = [k, v]
    c.pages = np.array([order], np.int32)
    c.pages_dev = dev(c.pages)
    c.desc = wq.kv_cache(k, v)
    check(c, lens, 2, queries(g, 1, 2, d), 0.125, with_acc=with_acc)


def test_shared_pages():
    """Two sequences over the same prefix page."""
    g = np.random.default_rng(16)
    lens = [40, 48]
    c = Cache(g, lens, 2, 64, "bf16", 16)
    c.pages[1, 0] = c.pages[0, 0]
    c.pages_dev = dev(c.pages)
    check(c, lens, 4, queries(g, 2, 4, 64), 0.125)


def test_calls_of_a_step_are_captured_in_a_graph():
    """Append, attention and eviction allocate nothing and do not synchronise: a captured
    step replays to the same bits."""
    g = np.random.default_rng(17)
    lens = [300, 41]
    c = Cache(g, lens, 2, 64, "bf16", 16)
    n, hq, cap = 2, 4, c.max_pages * 16
    x = torch.randn(n, (hq + 4) * 64, generator=torch.Generator().manual_seed(1)).cuda()
    table = torch.empty(512 * 64, device="cuda")
    wq.check(wq.wq_rope_table(512, 64, 10000.0, None, table))
    slot = dev(np.array([x - 1 for x in lens], np.int32))
    q, out = (torch.zeros(n, hq * 64, device="cuda") for _ in range(2))
    acc0 = torch.rand(n, 2, cap, generator=torch.Generator().manual_seed(2)).cuda()
    acc, acc2 = torch.zeros_like(acc0), torch.zeros_like(acc0)
    pos = torch.arange(cap, dtype=torch.int32, device="cuda").expand(n, 2, cap).contiguous()
    pos2, lensd = torch.zeros_like(pos), dev(np.array(lens, np.int32))
    lens2 = torch.zeros_like(lensd)
    size = max(wq.wq_attn_paged_workspace_bytes(c.desc, n, hq, c.max_pages, True),
               wq.wq_kv_evict_workspace_bytes(c.desc, n, c.max_pages, 200))
    room = workspace(size)

    full = [p.clone() for p in c.pools]

    def step(stream):
        acc.copy_(acc0)
        for p, p0 in zip(c.pools, full):  # the eviction moves rows
            p.copy_(p0)
        wq.check(wq.wq_kv_append(c.desc, n, hq, 64, 0, x, 8 * 64, x[:, hq * 64:], 8 * 64,
                                 x[:, (hq + 2) * 64:], 8 * 64, slot, table, 512, n, None, slot,
                                 c.pages_dev, c.max_pages, q, hq * 64, acc, pos, cap, stream=stream))
        wq.check(wq.wq_attn_paged(c.desc, n, hq, 0.125, 0, q, hq * 64, c.pages_dev, c.max_pages,
                                  lensd, None, 0, out, hq * 64, None, acc, acc, cap, room, size,
                                  stream=stream))
        wq.check(wq.wq_kv_evict(c.desc, n, c.pages_dev, c.max_pages, lensd, lensd, 200, 2, 50, acc,
                                pos, acc2, pos2, cap, lens2, room, size, stream=stream))

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(side)
    torch.cuda.synchronize()
    want = [t.clone() for t in (q, out, acc, acc2, pos2, lens2, *c.pools)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(side)
    for _ in range(3):
        for t in (q, out, acc2, pos2, lens2):
            t.zero_()
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip((q, out, acc, acc2, pos2, lens2, *c.pools), want):
        assert np.array_equal(bits(a), bits(b))
    assert lens2.tolist() == [200, 41]


@pytest.mark.parametrize("n,hq,long", [(300, 6, 30000), (60, 8, 40000), (3, 6, 50000)])
@pytest.mark.parametrize("with_acc", [False, True])
def test_one_long_row_among_short_ones(n, hq, long, with_acc):
    """The long rows are in dozens of parts, the others whole or in two: more rows than CTAs,
    fewer, few."""
    g = np.random.default_rng(n)
    lens = [int(x) for x in g.integers(0, 6, n)]
    lens[n // 2] = long
    c = Cache(g, lens, 2, 64, "bf16", 64, max_pages=-(-long // 64))
    check(c, lens, hq, queries(g, n, hq, 64), 0.125, with_acc=with_acc)


@pytest.mark.parametrize("n,length,hq,hkv,d,kind", [
    (1, 20000, 5, 1, 64, "bf16"),     # one row in hundreds of parts
    (2, 9000, 40, 1, 64, "f16"),      # and several tiles of heads to a group
    (1, 9000, 34, 2, 128, "f32"),
    (90, 200, 20, 1, 128, "bf16"),    # short caches, a group of more heads than in flight
    (40, 700, 33, 1, 64, "f16")])
@pytest.mark.parametrize("masked", [False, True])
def test_weights_of_large_groups(n, length, hq, hkv, d, kind, masked):
    g = np.random.default_rng(length + hq)
    lens = [length] + [int(x) for x in g.integers(length // 2, length, n - 1)]
    c = Cache(g, lens, hkv, d, kind, 16)
    cap = c.max_pages * 16
    mask = None
    if masked:
        mask = np.where(g.random((n, cap)) < 0.3, -np.inf, 0.1).astype(np.float32)
        mask[-1, :cap // 2] = -np.inf
    acc_in = np.abs(g.standard_normal((n, hkv, cap))).astype(np.float32)
    check(c, lens, hq, queries(g, n, hq, d), d ** -0.5, window=length // 2 if masked else 0,
          mask=mask, acc_in=acc_in, with_acc=True)
