"""GPU parity of wq_kv_evict: which slots stay, where they move, and that nothing else is
touched.  Nothing is computed: every comparison is exact."""
import numpy as np
import pytest
import torch

import gemv_transformer_gb300 as wq
from helpers import dev, status_ok
from kv_helpers import Cache, bits, workspace
from oracle import kv as okv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from gemv_transformer_gb300 import build
    build.build()
    wq.load()
    yield
    status_ok()


def run_evict(c, lens, seen, keep, sinks, recent, acc, pos, in_place=False, times=1, stream=None):
    n = len(lens)
    k0, v0 = (p.cpu() for p in c.pools)
    stride = acc.shape[2]
    accd, posd = dev(acc), dev(pos)
    lensd = dev(np.asarray(lens, np.int32))
    acc_out = accd if in_place else torch.full_like(accd, 9.0)
    pos_out = posd if in_place else torch.full_like(posd, -9)
    lens_out = lensd if in_place else torch.full_like(lensd, -9)
    size = wq.wq_kv_evict_workspace_bytes(c.desc, n, c.max_pages, keep)
    room = workspace(size)
    seend = dev(np.asarray(seen, np.int32))
    torch.cuda.synchronize()
    for _ in range(times):
        wq.check(wq.wq_kv_evict(c.desc, n, c.pages_dev, c.max_pages, lensd, seend, keep, sinks,
                                recent, accd, posd, acc_out, pos_out, stride, lens_out, room, size,
                                stream=stream), "wq_kv_evict")
    torch.cuda.synchronize()
    kb, vb = (x.view(torch.int32 if x.dtype == torch.float32 else torch.int16).numpy()
              for x in (k0, v0))
    kw, vw, aw, pw, nw = okv.evict(kb, vb, c.pages, lens, seen, keep, sinks, recent, acc, pos)
    assert np.array_equal(lens_out.cpu().numpy(), nw)
    for got, want in ((c.pools[0], kw), (c.pools[1], vw)):
        got = got.cpu()
        got = got.view(torch.int32 if got.dtype == torch.float32 else torch.int16).numpy()
        assert np.array_equal(got, want)
    a, p = acc_out.cpu().numpy(), pos_out.cpu().numpy()
    for s in range(n):
        m = nw[s]
        assert np.array_equal(a[s, :, :m].view(np.int32), aw[s, :, :m].view(np.int32))
        assert np.array_equal(p[s, :, :m], pw[s, :, :m])
        if not in_place:
            assert (a[s, :, m:] == 9.0).all() and (p[s, :, m:] == -9).all()
        else:
            assert np.array_equal(a[s, :, m:].view(np.int32), acc[s, :, m:].view(np.int32))
            assert np.array_equal(p[s, :, m:], pos[s, :, m:])
    status_ok()


def sums(g, n, h, cap, how="real"):
    if how == "ties":
        return g.integers(0, 4, (n, h, cap)).astype(np.float32)
    return np.exp(2 * g.standard_normal((n, h, cap))).astype(np.float32)


def positions(g, n, h, cap, seen):
    return np.stack([np.stack([g.choice(max(cap, seen[s]), cap, replace=False)
                               for _ in range(h)]) for s in range(n)]).astype(np.int32)


@pytest.mark.parametrize("kind,d,page,major", [("bf16", 128, 16, "head"), ("f16", 64, 1, "token"),
                                               ("f32", 256, 7, "gap"), ("bf16", 72, 64, "token"),
                                               ("f32", 8, 100, "head")])
@pytest.mark.parametrize("keep,sinks,recent", [(64, 4, 16), (1, 0, 0), (1, 0, 1), (100, 0, 100),
                                               (300, 4, 0), (199, 1, 50), (257, 0, 3)])
@pytest.mark.parametrize("how", ["real", "ties"])
def test_budgets(kind, d, page, major, keep, sinks, recent, how):
    g = np.random.default_rng(keep * 7 + d)
    lens = [0, 1, 64, 65, 200, 301, 512]
    c = Cache(g, lens, 2, d, kind, page, major, fill=1.0)
    cap = c.max_pages * page
    seen = [max(1, x) for x in lens]
    pos = np.tile(np.arange(cap, dtype=np.int32), (len(lens), 2, 1))
    run_evict(c, lens, seen, keep, sinks, recent, sums(g, len(lens), 2, cap, how), pos,
              in_place=keep % 2 == 0)


@pytest.mark.parametrize("length,keep", [(2049, 2048), (5000, 1), (5000, 4999), (20000, 777),
                                         (70001, 30000), (150000, 149000)])
@pytest.mark.parametrize("how", ["real", "ties"])
def test_long_rows_scrambled_positions(length, keep, how):
    g = np.random.default_rng(length + keep)
    lens = [length, length - 3]
    c = Cache(g, lens, 1, 8, "bf16", 64, fill=1.0)
    cap = c.max_pages * 64
    seen = [length + 500] * 2
    run_evict(c, lens, seen, keep, min(2, keep - 1), keep // 4, sums(g, 2, 1, cap, how),
              positions(g, 2, 1, cap, seen), in_place=how == "ties")


def test_many_rows():
    g = np.random.default_rng(3)
    lens = [int(x) for x in g.integers(0, 200, 90)]
    c = Cache(g, lens, 8, 8, "bf16", 16, fill=1.0)
    cap = c.max_pages * 16
    pos = np.tile(np.arange(cap, dtype=np.int32), (90, 8, 1))
    run_evict(c, lens, lens, 100, 2, 10, sums(g, 90, 8, cap), pos)


def test_special_weights():
    """NaN, infinities, both zeros, negatives, subnormals, everything equal."""
    g = np.random.default_rng(4)
    lens = [300] * 5
    c = Cache(g, lens, 1, 64, "bf16", 16, fill=1.0)
    cap = c.max_pages * 16
    acc = sums(g, 5, 1, cap)
    acc[0, 0, ::3] = np.nan
    acc[1, 0, ::5], acc[1, 0, 1::5], acc[1, 0, 2::5] = np.inf, -np.inf, -1.0
    acc[2, 0, :] = 0.5
    acc[3, 0, :] = np.where(g.random(cap) < 0.5, 0.0, -0.0)
    acc[4, 0, :] = g.integers(0, 3, cap) * np.float32(1e-45)
    pos = np.tile(np.arange(cap, dtype=np.int32), (5, 1, 1))
    for keep in (20, 150, 220):
        run_evict(c, lens, lens, keep, 3, 5, acc, pos)


def test_more_held_than_the_budget():
    """Repeated positions: sinks and recent slots beyond the budget, the lower ones stay."""
    g = np.random.default_rng(5)
    lens = [200]
    c = Cache(g, lens, 2, 64, "bf16", 16, fill=1.0)
    cap = c.max_pages * 16
    pos = np.zeros((1, 2, cap), np.int32)
    run_evict(c, lens, [200], 50, 1, 4, sums(g, 1, 2, cap), pos)


def test_again_on_the_same_arguments_is_the_same():
    """Out of place, a second call moves the same slots to the same places."""
    g = np.random.default_rng(6)
    lens = [500, 90]
    c = Cache(g, lens, 2, 64, "bf16", 16, fill=1.0)
    cap = c.max_pages * 16
    pos = np.tile(np.arange(cap, dtype=np.int32), (2, 2, 1))
    run_evict(c, lens, lens, 64, 4, 16, sums(g, 2, 2, cap), pos, times=3,
              stream=torch.cuda.Stream())


def test_lengths_and_pages_out_of_range():
    g = np.random.default_rng(7)
    lens = [64, 64, -3]
    c = Cache(g, lens, 1, 64, "bf16", 16, fill=1.0)
    c.pages[1, 3] = 10 ** 6
    c.pages[0, 1] = -1
    c.pages_dev = dev(c.pages)
    acc = sums(g, 3, 1, 64)
    pos = np.tile(np.arange(64, dtype=np.int32), (3, 1, 1))
    before = [p.clone() for p in c.pools]
    accd, posd = dev(acc), dev(pos)
    a, p = torch.zeros_like(accd), torch.zeros_like(posd)
    n = torch.full((3,), -9, dtype=torch.int32, device="cuda")
    size = wq.wq_kv_evict_workspace_bytes(c.desc, 3, 4, 32)
    wq.check(wq.wq_kv_evict(c.desc, 3, c.pages_dev, 4, dev(np.array([9999, 64, -3], np.int32)),
                            dev(np.array([64, 64, 1], np.int32)), 32, 0, 0, accd, posd, a, p, 64,
                            n, workspace(size), size))
    torch.cuda.synchronize()
    assert wq.wq_get_device_status() == wq.WQ_ERR_BAD_INDEX
    assert n.tolist() == [32, 32, 0]
    zero = np.zeros((1, 1, 64, 1), np.int16)  # weights and positions move all the same
    for s in (0, 1):
        _, _, aw, pw, _ = okv.evict(zero, zero, np.zeros((1, 1), np.int32), [64], [64], 32, 0, 0,
                                    acc[s:s + 1], pos[s:s + 1])
        assert np.array_equal(a[s, 0, :32].cpu().numpy(), aw[0, 0, :32])
        assert np.array_equal(p[s, 0, :32].cpu().numpy(), pw[0, 0, :32])
    live = set(c.pages[c.pages >= 0].tolist()) - {10 ** 6}
    for now, was in zip(c.pools, before):
        rest = [i for i in range(now.shape[0]) if i not in live]
        assert np.array_equal(bits(now[rest]), bits(was[rest]))


def test_cache_beyond_4_gib():
    page, d, step, count = 16, 64, (1 << 30) + 64, 5
    room = torch.empty(count * step, dtype=torch.bfloat16, device="cuda")
    k = room.as_strided((count, 1, page, d), (step, page * d, d, 1))
    v = room[4096:].as_strided((count, 1, page, d), (step, page * d, d, 1))
    g = np.random.default_rng(8)
    x = torch.from_numpy(g.standard_normal((2, 80, d)).astype(np.float32)).bfloat16()
    order = [4, 0, 3, 1, 2]
    for i, p in enumerate(order):
        k[p, 0], v[p, 0] = x[0, 16 * i:16 * i + 16].cuda(), x[1, 16 * i:16 * i + 16].cuda()
    acc = sums(g, 1, 1, 80)
    pos = np.arange(80, dtype=np.int32).reshape(1, 1, 80)
    accd, posd, lens = dev(acc), dev(pos), dev(np.array([80], np.int32))
    cache = wq.kv_cache(k, v)
    size = wq.wq_kv_evict_workspace_bytes(cache, 1, 5, 20)
    wq.check(wq.wq_kv_evict(cache, 1, dev(np.array([order], np.int32)), 5, lens, lens, 20, 0, 0,
                            accd, posd, accd, posd, 80, lens.clone(), workspace(size), size))
    torch.cuda.synchronize()
    at = posd[0, 0, :20].cpu().long()
    assert sorted(at.tolist()) == sorted(np.argsort(-acc[0, 0], kind="stable")[:20].tolist())
    for pool, want in ((k, x[0]), (v, x[1])):
        got = torch.cat([pool[order[0], 0], pool[order[1], 0]])[:20].cpu()
        assert torch.equal(got, want[at])


@pytest.mark.parametrize("n,hkv,length,keep,d,kind", [
    (1, 1, 400000, 250000, 8, "bf16"),   # longer than eight CTAs' key arrays hold
    (1, 1, 350001, 350000, 8, "bf16"),
    (2, 1, 20000, 9000, 128, "f32"),     # few rows, many bytes: moved by all SMs
    (1, 3, 30000, 12000, 256, "f16"),
    (2, 2, 70000, 30000, 64, "bf16")])
@pytest.mark.parametrize("ties", [False, True])
def test_long_rows_by_their_own_numbers(n, hkv, length, keep, d, kind, ties):
    """Rows that hold their slot's number: each survivor is where the rule puts it."""
    page = 64
    pages = -(-length // page)
    g = np.random.default_rng(length + ties)
    table = np.stack([g.permutation(pages) + s * pages for s in range(n)]).astype(np.int32)
    from kv_helpers import TYPES
    shape = (n * pages, hkv, page, d)
    k = torch.zeros(shape, dtype=TYPES[kind], device="cuda")
    bits_of = {2: torch.int16, 4: torch.int32}[k.element_size()]
    number = torch.arange(pages * page, device="cuda")
    for s in range(n):
        at = torch.from_numpy(table[s]).cuda().long()
        low, high = (number & 0x7FFF).view(pages, page), (number >> 15).view(pages, page)
        for h in range(hkv):  # the first two values are the slot's number
            k.view(bits_of)[at, h, :, 0] = low.to(bits_of)
            k.view(bits_of)[at, h, :, 1] = high.to(bits_of)
    v = k.clone()
    acc = g.integers(0, 50, (n, hkv, length)).astype(np.float32) if ties else \
        np.exp(2 * g.standard_normal((n, hkv, length))).astype(np.float32)
    pos = np.broadcast_to(np.arange(length, dtype=np.int32), (n, hkv, length)).copy()
    accd, posd = dev(acc), dev(pos)
    lens = dev(np.full(n, length, np.int32))
    cache = wq.kv_cache(k, v)
    size = wq.wq_kv_evict_workspace_bytes(cache, n, pages, keep)
    torch.cuda.synchronize()
    wq.check(wq.wq_kv_evict(cache, n, dev(table), pages, lens, lens.clone(), keep, 3, 500, accd, posd,
                            accd, posd, length, lens, workspace(size), size))
    torch.cuda.synchronize()
    status_ok()
    assert lens.tolist() == [keep] * n
    for s in range(n):
        rows = torch.from_numpy(table[s]).cuda().long()
        for h in range(hkv):
            rank = np.where((pos[s, h] < 3) | (pos[s, h] >= length - 500), np.inf, acc[s, h])
            stay = np.zeros(length, bool)
            stay[np.argsort(-rank, kind="stable")[:keep]] = True
            want = np.arange(keep)
            want[~stay[:keep]] = keep + np.flatnonzero(stay[keep:])
            assert np.array_equal(posd[s, h, :keep].cpu().numpy(), want)
            assert np.array_equal(accd[s, h, :keep].cpu().numpy(), acc[s, h][want])
            for pool in (k, v):
                row = pool.view(bits_of)[rows, h].view(-1, d)[:keep].long()
                assert np.array_equal((row[:, 0] + (row[:, 1] << 15)).cpu().numpy(), want)
                assert not row[:, 2:].any()


@pytest.mark.parametrize("n,h,keep,d,kind,page,major", [
    (1, 1, 1, 64, "bf16", 1, "head"), (3, 2, 255, 128, "f16", 7, "gap"),
    (70, 8, 300, 8, "bf16", 64, "token"),   # short rows, more than two per SM
    (1, 2, 6000, 256, "f32", 100, "head"),  # two, four and eight CTAs to a row
    (2, 1, 12001, 72, "bf16", 64, "token"), (1, 1, 30000, 8, "f32", 64, "head")])
@pytest.mark.parametrize("how", ["real", "equal", "nan", "held", "last"])
def test_one_over_the_budget(n, h, keep, d, kind, page, major, how):
    """The least slot goes, of equal ones the highest, and the last takes its place; rows at
    and below the budget are among them."""
    g = np.random.default_rng(keep + d)
    lens = [keep + 1 if s % 3 != 2 else keep - s % 2 for s in range(n)]
    c = Cache(g, lens, h, d, kind, page, major, fill=1.0)
    cap = c.max_pages * page
    acc = sums(g, n, h, cap)
    pos = positions(g, n, h, cap, [keep + 9] * n)
    sinks, recent = min(2, keep), keep // 3
    if how == "equal":
        acc[:] = 0.25
    elif how == "nan":
        acc[:, :, g.integers(0, cap, 3)] = np.nan
        acc[:, :, g.integers(0, cap, 3)] = -np.inf
    elif how == "held":  # more than the budget: the highest slot goes
        pos[:] = g.integers(0, 2, pos.shape)
    elif how == "last":  # nothing moves
        acc[:, :, keep] = -1.0
        pos[:, :, keep] = sinks
    seen = [max(keep + 9, cap)] * n
    run_evict(c, lens, seen, keep, sinks, recent, acc, pos, in_place=how in ("real", "held"))


def test_one_over_with_pages_out_of_range():
    """The last slot's page, then the page of the slot that goes: neither is read or written."""
    g = np.random.default_rng(9)
    c = Cache(g, [65, 65], 1, 64, "bf16", 16, fill=1.0)
    c.pages[0, 4] = -1
    c.pages[1, 1] = 10 ** 6
    c.pages_dev = dev(c.pages)
    acc = 1 + sums(g, 2, 1, 80)
    acc[:, :, 20] = 0.5
    pos = np.tile(np.arange(80, dtype=np.int32), (2, 1, 1))
    before = [p.clone() for p in c.pools]
    accd, posd = dev(acc), dev(pos)
    lens = dev(np.array([65, 65], np.int32))
    size = wq.wq_kv_evict_workspace_bytes(c.desc, 2, 5, 64)
    wq.check(wq.wq_kv_evict(c.desc, 2, c.pages_dev, 5, lens, lens.clone(), 64, 0, 0, accd, posd,
                            accd, posd, 80, lens, workspace(size), size))
    torch.cuda.synchronize()
    assert wq.wq_get_device_status() == wq.WQ_ERR_BAD_INDEX
    assert lens.tolist() == [64, 64]
    for now, was in zip(c.pools, before):
        assert np.array_equal(bits(now), bits(was))
    assert (accd[:, 0, 20].cpu().numpy() == acc[:, 0, 64]).all()
    assert (posd[:, 0, 20] == 64).all()
