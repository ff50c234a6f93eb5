"""The calls for several new tokens per sequence as they are used together, step after step, and
what they promise when a wait runs out, when `starts` overlap, and on two streams.

Tolerances.  The append's are those of its own test: 2^-19 of the terms' magnitude and half a step.
The attention's and accept's are checked against the device's own q and caches, which a step reads:
those of tests/test_attn_tokens_gpu.py, and whole numbers."""
import numpy as np
import pytest
import torch

import gemv_transformer_gb300 as wq
from helpers import dev, status_ok
from kv_helpers import Cache, bits, workspace
from oracle import tokens as ot
from test_attn_tokens_gpu import U, Case
from tokens_helpers import HALF, KINDS, TORCH, angles, random_tree, tree_words

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from gemv_transformer_gb300 import build
    build.build()
    wq.load()
    yield
    status_ok()


class Steps:
    """Layers of one form over n sequences' pages; a prompt, then steps of drafted trees."""

    def __init__(self, seed, kind, qtype, hq=4, hkv=2, d=64, layers=2, n=3, page=16, wide=20):
        self.g = np.random.default_rng(seed)
        self.kind, self.qtype, self.hq, self.hkv, self.d = kind, qtype, hq, hkv, d
        self.n, self.page, self.wide = n, page, wide
        pages = self.g.permutation(n * wide + 2)[:n * wide].reshape(n, wide).astype(np.int32)
        self.pages, self.pages_dev = pages, dev(pages)
        self.pools = [[torch.full((n * wide + 2, hkv, page, d), float("nan"), dtype=TORCH[kind],
                                  device="cuda") for _ in range(2)] for _ in range(layers)]
        self.caches = wq.kv_caches(*zip(*self.pools))
        w = [dev((1 + 0.2 * self.g.standard_normal(d)).astype(np.float32)) for _ in range(2)]
        self.weights = w
        self.norms = [wq.head_norm(ot.RMS, 1e-6, x) for x in w]
        self.table = angles(wide * page, d // 2)
        self.table_dev = dev(self.table)
        self.lens = torch.zeros(n, dtype=torch.int32, device="cuda")

    def host(self, layer):
        return [p.double().cpu().numpy() for p in self.pools[layer]]

    def step(self, counts, trees=None):
        """Append and attend in every layer; parents and above[] of each sequence's nodes."""
        g, n, d, hq, hkv = self.g, self.n, self.d, self.hq, self.hkv
        m = sum(counts)
        starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        seq = np.repeat(np.arange(n), counts).astype(np.int32)
        node = np.concatenate([np.arange(c) for c in counts]).astype(np.int32)
        depth = node.copy() if trees is None else np.concatenate(
            [[len(a) - 1 for a in above] for _, above in trees]).astype(np.int32)
        before = self.lens.cpu().numpy()
        self.lens += dev(np.array(counts, np.int32))
        slot, pos = before[seq] + node, (before[seq] + depth).astype(np.int32)
        pos2 = np.stack([pos, pos // 2]).astype(np.int32)
        seq_d, slot_d, pos_d, starts_d = (dev(x) for x in (seq, slot.astype(np.int32), pos2, starts))
        rope = wq.rope_axes(d, 0, [d // 4, d // 4], pos_d, self.table_dev)
        above = None if trees is None else [a for _, rows in trees for a in rows]
        words = None if trees is None else tree_words(above, -(-max(counts) // 32))
        form = None if trees is None else wq.attn_form(tree=words, pos=pos_d)
        size = wq.wq_attn_tokens_workspace_bytes(self.caches[0], n, m, hq, KINDS[self.qtype])
        room, wide = workspace(size), (hq + 2 * hkv) * d
        for i, cache in enumerate(self.caches):
            qkv = dev(g.standard_normal((m, wide)).astype(np.float32))
            q = torch.empty(m, hq * d, dtype=TORCH[self.qtype], device="cuda")
            out = torch.empty_like(q)
            wq.check(wq.wq_kv_append_norm(
                cache, m, hq, *self.norms, rope, qkv, wide, qkv[:, hq * d:], wide,
                qkv[:, (hq + hkv) * d:], wide, n, seq_d, slot_d, self.pages_dev, self.wide,
                KINDS[self.qtype], q, hq * d, None, None, 0))
            wq.check(wq.wq_attn_tokens(
                cache, n, m, hq, d ** -0.5, form, KINDS[self.qtype], q, hq * d, starts_d,
                self.pages_dev, self.wide, self.lens, KINDS[self.qtype], out, hq * d, None, room,
                size))
            self.check(i, qkv, q, out, seq, slot, pos2, starts, above, pos)
        return starts, starts_d

    def check(self, i, qkv, q, out, seq, slot, pos, starts, above, own_pos):
        m, d, hq, hkv = len(seq), self.d, self.hq, self.hkv
        x = qkv.double().cpu().numpy().reshape(m, -1, d)
        cs = ot.cos_sin([d // 4, d // 4], pos, self.table.astype(np.float64))
        got_q = q.double().cpu().numpy().reshape(m, hq, d)
        k, v = self.host(i)
        where = self.pages[seq, slot // self.page], slot % self.page
        for w, part, got, kind in ((0, x[:, :hq], got_q, self.qtype),
                                   (1, x[:, hq:hq + hkv], k[where[0], :, where[1]], self.kind)):
            y, mag = ot.norm(part, ot.RMS, float(np.float32(1e-6)), self.weights[w].cpu().numpy())
            y, mag = ot.turn(y, cs, mag=mag)
            tol = 2.0 ** -19 * mag
            assert (np.abs(got - y) <= tol + HALF[kind] * (np.abs(y) + tol)).all()
        rounded = qkv.view(m, -1, d)[:, hq + hkv:].to(TORCH[self.kind]).double().cpu().numpy()
        assert (v[where[0], :, where[1]] == rounded).all()
        lens = self.lens.cpu().numpy()
        r = ot.attention(got_q, k, v, self.pages, starts, lens, d ** -0.5, tree=above,
                         pos=None if above is None else own_pos)
        got = out.double().cpu().numpy().reshape(m, hq, d)
        ex = (d + 8) * U * r["sx"] + 8 * U * r["mx"]
        tol = (2 * ex + (r["n"][:, None] + 80) * U)[..., None] * r["pv"]
        if self.qtype != "f32":
            tol = tol + HALF[self.qtype] * r["pv"]
            if self.qtype == "f16":
                tol = tol + 2.0 ** -22 * r["n"][:, None, None] * r["pv"].max(-1, keepdims=True)
            tol = tol + HALF[self.qtype] * (np.abs(r["out"]) + tol) + 2.0 ** -25
        assert (np.abs(got - r["out"]) <= tol).all()


@pytest.mark.parametrize("kind,qtype", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"),
                                        ("f32", "f32")])
@pytest.mark.parametrize("hq,hkv,d,page", [(4, 2, 64, 16), (6, 1, 128, 8), (3, 3, 32, 7),
                                           (4, 1, 256, 32)])
def test_prompt_then_drafted_steps(kind, qtype, hq, hkv, d, page):
    s = Steps(1, kind, qtype, hq, hkv, d, page=page, wide=-(-300 // page))
    g = s.g
    s.step([70, 1, 150])          # prompts
    s.step([20, 30, 1])           # pieces
    for counts in ([16, 1, 40], [5, 33, 2], [8, 8, 8]):
        trees = [random_tree(g, c) for c in counts]
        starts, starts_d = s.step(counts, trees)
        m = sum(counts)
        parent = np.concatenate([p for p, _ in trees]).astype(np.int32)
        tokens, choice = (g.integers(0, 3, m).astype(np.int32) for _ in range(2))
        lens = s.lens.cpu().numpy()
        before = [s.host(i) for i in range(2)]
        f = dict(dtype=torch.int32, device="cuda")
        path, accepted, nxt, new = (torch.full((x,), 77, **f) for x in (m, s.n, s.n, s.n))
        wq.check(wq.wq_kv_accept(s.caches, s.n, m, s.pages_dev, s.wide, starts_d, dev(parent),
                                 dev(tokens), dev(choice), s.lens, path, accepted, nxt, new))
        want = ot.accept(starts, parent, tokens, choice, lens)
        for got, w in zip((path, accepted, nxt, new), want):
            assert got.cpu().numpy().tolist() == np.asarray(w).tolist()
        for i in range(2):
            for old, now in zip(before[i], s.host(i)):
                for q, nodes in enumerate(want[4]):
                    base = lens[q] - counts[q]
                    for j, x in enumerate(nodes):
                        a, b = base + x, base + j
                        assert (now[s.pages[q, b // page], :, b % page]
                                == old[s.pages[q, a // page], :, a % page]).all()
        s.lens = new              # the next step goes on behind the accepted paths
    # A decode step over what is left agrees with a call of one token to a sequence.
    s.step([1, 1, 1])


def overlapping(kind, qtype, n=40, rows=60, hq=4, d=64):
    g = np.random.default_rng(3)
    cache = Cache(g, [rows] * n, 2, d, kind)
    starts = dev(np.array([0, rows] * (n // 2) + [0], np.int32))
    q = torch.randn(rows, hq * d, device="cuda").to(TORCH[qtype])
    return cache, starts, q, dev(np.full(n, rows, np.int32))


@pytest.mark.parametrize("kind,qtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_overlapping_starts_stay_in_the_workspace(kind, qtype):
    """Ranges that hold more tokens than n_tok together: recorded, and nothing is written behind the
    workspace or the rows."""
    n, rows, hq, d = 40, 60, 4, 64
    cache, starts, q, lens = overlapping(kind, qtype, n, rows, hq, d)
    size = wq.wq_attn_tokens_workspace_bytes(cache.desc, n, rows, hq, KINDS[qtype])
    room = torch.full((size + (1 << 20),), 0x5A, dtype=torch.uint8, device="cuda")
    out = torch.full((rows + 8, hq * d), 9.0, dtype=TORCH[qtype], device="cuda")
    wq.check(wq.wq_attn_tokens(cache.desc, n, rows, hq, 0.1, None, KINDS[qtype], q, hq * d, starts,
                               cache.pages_dev, cache.max_pages, lens, KINDS[qtype], out, hq * d,
                               None, room, size))
    assert wq.wq_get_device_status() == wq.WQ_ERR_BAD_INDEX
    assert (room[size:] == 0x5A).all()
    assert (out[rows:] == 9).all() and torch.isfinite(out.float()).all()
    Case(4, [30, 3], [60, 10], hq, 2, d, kind, qtype).run().check()


@pytest.mark.parametrize("kind,qtype", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"),
                                        ("f32", "f32"), ("f16", "f32")])
def test_scores_that_are_not_numbers_reach_the_lse(kind, qtype):
    """A query of NaN, and one against keys of which one is NaN: out and lse are NaN there only."""
    c = Case(5, [40, 9], [300, 0], 4, 2, 64, kind, qtype)
    c.q[3, 64:128] = float("nan")
    c.run()
    got = c.out.double().cpu().numpy()[:c.m].reshape(c.m, 4, 64)
    lse = c.lse.cpu().numpy()[:c.m]
    bad = np.zeros((c.m, 4), bool)
    bad[3, 1] = True
    assert (np.isnan(lse) == bad).all() and (np.isnan(got) == bad[..., None]).all()


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("cap", [300.0, 20000.0])
def test_large_caps_of_16_bit_queries(kind, cap):
    """The cap's own error is relative there, 8 2^-24 of a score; the fast one's would be 2^-22 of
    the cap."""
    c = Case(6, [40, 150], [90, 20], 4, 2, 64, kind, kind, softcap=cap, qscale=20.0, otype="f32")
    w = c.run().want()
    ex = (c.d + 8) * U * w["sx"] + 16 * U * w["mx"]
    tol = ex + (w["n"][:, None] + 16) * U + 4 * U * np.abs(w["lse"])
    assert (np.abs(c.lse.double().cpu().numpy()[:c.m] - w["lse"]) <= tol).all()


@pytest.mark.parametrize("kind,qtype,counts,page,d", [
    (kind, qtype, counts, page, 128) for page in (16, 7) for kind, qtype, counts in
    (("bf16", "bf16", [200, 500]), ("bf16", "bf16", [16, 9]), ("bf16", "f32", [16, 9]),
     ("f16", "f16", [300, 40]))] + [("bf16", "bf16", [200, 500], 16, 256)])
def test_wait_limit_expires_without_hang(kind, qtype, counts, page, d):
    """A one-poll limit makes the first wait that finds nothing give up: the call records it, drains
    its copies and returns; the next one is right."""
    c = Case(7, counts, [900, 1500], 8, 2, d, kind, qtype, page=page)
    seen = []
    wq.wq_set_wait_limit(1)
    try:
        for _ in range(5):
            c.run()
            seen.append(wq.wq_get_device_status())
            if seen[-1] == wq.WQ_ERR_DEVICE_TIMEOUT:
                break
    finally:
        wq.wq_set_wait_limit(0)
    assert wq.WQ_ERR_DEVICE_TIMEOUT in seen
    assert wq.wq_get_device_status() == wq.WQ_OK
    c.run().check()


@pytest.mark.parametrize("kind,qtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_two_streams_with_workspaces_of_their_own(kind, qtype):
    a = Case(8, [64, 9], [700, 40], 8, 2, 128, kind, qtype).run()
    b = Case(9, [300], [100], 8, 2, 128, kind, qtype).run()
    want = a.out.clone(), b.out.clone()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(6):
        for c, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                c.run(c.out, c.lse, None, c.room)
    torch.cuda.synchronize()
    assert torch.equal(a.out, want[0]) and torch.equal(b.out, want[1])
    a.check(), b.check()


@pytest.mark.parametrize("kind,qtype", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"),
                                        ("f32", "f32")])
@pytest.mark.parametrize("counts,contexts,hq,hkv,d", [
    ([700], [2000], 12, 4, 64),       # groups of 3: queries row by row
    ([900, 40], [10, 3000], 8, 8, 128),   # parts joined by the last of their CTAs
    ([2500], [0], 2, 1, 64),
    ([3] * 40, [400] * 40, 130, 1, 64),   # more heads than a row tile
    ([300, 5], [40, 900], 8, 4, 256), ([200], [30], 3, 1, 136), ([30, 1] * 9, [300] * 18, 16, 8, 192)])
def test_shapes_of_the_deal(kind, qtype, counts, contexts, hq, hkv, d):
    Case(10, counts, contexts, hq, hkv, d, kind, qtype, page=32).run().check()


@pytest.mark.parametrize("kind,qtype", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"),
                                        ("f32", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("d", [64, 200])
def test_bits_depend_on_nothing_that_is_not_seen(kind, qtype, tree, d):
    """Other sequences' queries and caches, rows behind the last sequence and slots that a token does
    not see: NaN or large, they change no bit."""
    c = Case(12, [40, 170], [90, 300], 4, 2, d, kind, qtype, tree=tree, extra=9).run()
    first = c.out.clone(), c.lse.clone()
    c.q[40:] = float("nan")                    # the second sequence and the rows behind
    c.out.fill_(9), c.lse.fill_(9)
    c.run(c.out, c.lse)
    assert torch.equal(c.out[:40], first[0][:40]) and torch.equal(c.lse[:40], first[1][:40])
    c = Case(12, [40, 170], [90, 300], 4, 2, d, kind, qtype, tree=tree, extra=9)
    for value in (float("nan"), 1e4, float("inf")):
        for s, j in ((0, 90 + 30), (1, 300 + 150), (1, 300 + 100)):
            for pool in c.cache.pools:
                pool[int(c.cache.pages[s, j // 16]), :, j % 16] = value
        c.run()
        for t in range(c.m):
            s = int(t >= 40)
            j = t - 40 * s
            hidden = [30] if s == 0 else [150, 100]
            sees = [b for b in hidden if (b in c.tree[t] if tree else b <= j)]
            if not sees:
                assert torch.equal(c.out[t], first[0][t]) and torch.equal(c.lse[t], first[1][t]), t


@pytest.mark.parametrize("page,major", [(7, "head"), (8, "gap"), (24, "token"), (100, "head")])
def test_pages_of_wide_heads(page, major):
    for kind in ("bf16", "f16"):
        Case(13, [20, 35], [210, 91], 4, 2, 256, kind, kind, page, major).run().check()
        Case(14, [20, 35], [210, 91], 4, 2, 136, kind, kind, page, major, tree=True).run().check()


def test_workspaces_cover_what_is_asked():
    """No more bytes are touched than the size says, for the sizes around a row tile."""
    for kind, qtype in (("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")):
        for count in (1, 31, 32, 33, 64, 65, 129):
            c = Case(11, [count, 1, count], [50, 0, 260], 8, 2, 64, kind, qtype)
            size = wq.wq_attn_tokens_workspace_bytes(c.cache.desc, 3, c.rows, 8, KINDS[qtype])
            room = torch.full((size + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
            c.run(room=room).check()
            assert (room[size:] == 0x5A).all()


def test_the_same_step_twice_gives_the_same_bits():
    runs = []
    for _ in range(2):
        s = Steps(2, "bf16", "bf16")
        s.step([40, 3, 17])
        s.step([16, 1, 7], [random_tree(np.random.default_rng(i), c) for i, c in
                            enumerate([16, 1, 7])])
        runs.append([bits(p) for pools in s.pools for p in pools])
    assert all((a == b).all() for a, b in zip(*runs))
