"""wq_kv_accept_slots: wq_kv_accept, and the slots' weights and positions moved with k and v.  Nothing is
computed: every comparison is exact."""
import numpy as np
import pytest
import torch

import gemv_transformer_gb300 as wq
from helpers import dev, status_ok
from kv_helpers import bits, workspace
from oracle import kv as okv
from oracle import tokens as ot
from test_kv_accept_gpu import Draft
from tokens_helpers import angles

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from gemv_transformer_gb300 import build
    build.build()
    wq.load()
    yield
    status_ok()


class Slots(Draft):
    """A draft with arrays of weights and positions in each layer; `without` have none."""

    def __init__(self, seed, counts, contexts, layers=2, hkv=2, d=64, kind="bf16", page=16, pad=3,
                 without=(), **kw):
        super().__init__(seed, counts, contexts, layers, hkv, d, kind, page, **kw)
        g = np.random.default_rng(seed + 100)
        self.hkv, self.n = hkv, len(counts)
        self.stride = self.pages.shape[1] * page + pad
        shape = (self.n, hkv, self.stride)
        self.acc = [None if (i, "acc") in without else g.random(shape, np.float32)
                    for i in range(layers)]
        self.pos = [None if (i, "pos") in without else
                    g.integers(-9, 10 ** 6, shape).astype(np.int32) for i in range(layers)]
        self.acc_dev, self.pos_dev = ([None if x is None else dev(x) for x in a]
                                      for a in (self.acc, self.pos))

    def call(self, outs, ins, one=False):
        arr = (wq.KvCache * len(self.caches))(*[c.desc for c in self.caches])
        return wq.wq_kv_accept_slots(
            self.caches[0].desc if one else arr, self.n, max(1, len(self.parent)), ins[0],
            self.pages.shape[1], *ins[1:], *outs,
            wq.slot_arrays(self.acc_dev[:1] if one else self.acc_dev,
                           self.pos_dev[:1] if one else self.pos_dev), self.stride)

    def inputs(self):
        some = [x if len(x) else np.zeros(1, np.int32)
                for x in (self.parent, self.tokens, self.choice)]
        return [dev(x) for x in (self.pages, self.starts, *some, self.lens)]

    def run(self, one=False):
        f = dict(device="cuda", dtype=torch.int32)
        self.path = torch.full((max(1, len(self.parent)) + 3,), 77, **f)
        self.accepted, self.next, self.lens_out = (torch.full((self.n + 2,), 77, **f)
                                                   for _ in range(3))
        wq.check(self.call([self.path, self.accepted, self.next, self.lens_out], self.inputs(), one))
        torch.cuda.synchronize()

    def check(self):
        count = super().check()  # outputs, and k and v of every layer
        nodes = ot.accept(self.starts, self.parent, self.tokens, self.choice, self.lens)[4]
        self.check_arrays(nodes)
        return count

    def check_arrays(self, nodes, skip=lambda s, slot: False):
        for olds, gots in ((self.acc, self.acc_dev), (self.pos, self.pos_dev)):
            for old, got in zip(olds, gots):
                if old is None:
                    continue
                want = old.copy()
                for s in range(self.n):
                    b = self.lens[s] - self.counts[s]
                    for i, node in enumerate(nodes[s]):
                        if not (skip(s, b + node) or skip(s, b + i)):
                            want[s, :, b + i] = old[s, :, b + node]
                assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("kind,page,major", [("bf16", 16, "head"), ("f16", 7, "token"),
                                             ("f32", 1, "gap"), ("bf16", 100, "head")])
@pytest.mark.parametrize("counts,contexts", [
    ([1], [0]), ([2], [5]), ([16], [100]), ([32, 0, 33, 1, 64], [0, 9, 31, 4, 100]),
    ([130, 7], [3, 50]), ([31, 65, 97], [1, 1, 1])])
def test_accept(kind, page, major, counts, contexts):
    Slots(1, counts, contexts, 2, 3, 40, kind, page, major=major).check()


def test_arrays_that_are_not_there():
    Slots(2, [40, 9], [7, 20], 3, without=[(0, "acc"), (1, "pos"), (2, "acc"), (2, "pos")]).check()


def test_many_layers_heads_and_sequences():
    g = np.random.default_rng(3)
    counts = [int(x) for x in g.integers(0, 6, 300)]
    Slots(3, counts, [int(x) for x in g.integers(0, 9, 300)], 2, 1, 8, "f32", 4).check()
    Slots(4, [9, 20], [10, 3], 53, 1, 16, pad=0).check()  # more layers than one launch takes
    Slots(5, [9, 20], [10, 3], 2, 300, 8).check()


def test_agrees_with_the_call_without_arrays():
    a, b = Draft(6, [24, 50], [30, 8], 2), Slots(6, [24, 50], [30, 8], 2)
    a.run(), b.run()
    for x, y in zip(a.caches, b.caches):
        for p, q in zip(x.pools, y.pools):
            assert (bits(p) == bits(q)).all()
    for x, y in ((a.path, b.path), (a.accepted, b.accepted), (a.next, b.next),
                 (a.lens_out, b.lens_out)):
        assert torch.equal(x, y)


def test_captured():
    d = Slots(7, [24, 50], [30, 8])
    f = dict(device="cuda", dtype=torch.int32)
    outs = [torch.zeros(74, **f)] + [torch.zeros(2, **f) for _ in range(3)]
    ins = d.inputs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wq.check(d.call(outs, ins))
    graph.replay()
    torch.cuda.synchronize()
    d.check_arrays(ot.accept(d.starts, d.parent, d.tokens, d.choice, d.lens)[4])


def test_bad_indexes():
    """Refused sequences keep their arrays, and so does a node whose page is out of range; a length
    beyond the arrays is one beyond the pages."""
    d = Slots(8, [20, 30, 10, 5], [40, 12, 3, 2], agree=1.0)
    nodes = ot.accept(d.starts, d.parent, d.tokens, d.choice, d.lens)[4]
    d.lens[2], d.lens[3] = 10 ** 6, 4
    d.run()
    assert wq.wq_get_device_status() == wq.WQ_ERR_BAD_INDEX
    d.check_arrays(nodes[:2] + [[], []])
    d = Slots(9, [40], [40], agree=1.0, page=4)
    nodes = ot.accept(d.starts, d.parent, d.tokens, d.choice, d.lens)[4]
    assert len(nodes[0]) > 4  # so that the fifth node is on the page
    lost = (40 + nodes[0][4]) // 4
    d.pages = d.pages.copy()
    d.pages[0, lost] = -3
    d.run()
    assert wq.wq_get_device_status() == wq.WQ_ERR_BAD_INDEX
    d.check_arrays(nodes, lambda s, slot: slot // 4 == lost)
    d = Slots(10, [20, 30], [40, 12], pad=0, agree=1.0)
    nodes = ot.accept(d.starts, d.parent, d.tokens, d.choice, d.lens)[4]
    d.stride = 59  # sequence 0 has 60 slots
    d.acc, d.pos = ([x[:, :, :59].copy() for x in a] for a in (d.acc, d.pos))
    d.acc_dev, d.pos_dev = ([dev(x) for x in a] for a in (d.acc, d.pos))
    d.run()
    assert wq.wq_get_device_status() == wq.WQ_ERR_BAD_INDEX
    assert d.accepted.tolist()[:2] == [0, len(nodes[1])] and d.lens_out.tolist()[0] == 60
    d.check_arrays([[], nodes[1]])


def test_a_step_of_drafts_before_an_eviction():
    """Append with positions, accept, evict: the accepted slots have the positions of their tokens,
    and the eviction keeps the newest of them."""
    context, hkv, d, page = 40, 2, 64, 8
    draft = Slots(11, [24], [context], 1, hkv, d, page=page, agree=1.0)
    n = len(draft.parent)
    depth = []
    for p in draft.parent:
        depth.append(0 if p < 0 else depth[p] + 1)
    where = np.array([context + x for x in depth], np.int32)
    draft.pos[0][:, :, :context] = np.arange(context)
    draft.pos_dev = [dev(draft.pos[0])]
    x = torch.randn(n, 2 * hkv * d, device="cuda")
    pos, table = dev(where[None]), dev(angles(128, d // 2))
    wq.check(wq.wq_kv_append_norm(
        draft.caches[0].desc, n, 0, None, None, wq.rope_axes(d, 0, [d // 2], pos, table), None, 0,
        x, 2 * hkv * d, x[:, hkv * d:], 2 * hkv * d, 1, dev(np.zeros(n, np.int32)),
        dev(np.arange(context, context + n, dtype=np.int32)), dev(draft.pages),
        draft.pages.shape[1], wq.WQ_F32, None, 0, draft.acc_dev[0], draft.pos_dev[0], draft.stride))
    draft.run()
    count = int(draft.accepted[0])
    assert count > 3
    length = context + count
    got = draft.pos_dev[0].cpu().numpy()
    assert (got[0, :, :length] == np.arange(length)).all()
    c, keep, recent = draft.caches[0], 30, count + 5
    acc, lens = draft.acc_dev[0].cpu().numpy(), draft.lens_out[:1]
    ints = [p.cpu().view(torch.int16).numpy() for p in c.pools]
    want = okv.evict(*ints, draft.pages, [length], [length], keep, 2, recent, acc, got)
    size = wq.wq_kv_evict_workspace_bytes(c.desc, 1, draft.pages.shape[1], keep)
    room, lens_out = workspace(size), torch.zeros(1, dtype=torch.int32, device="cuda")
    wq.check(wq.wq_kv_evict(c.desc, 1, dev(draft.pages), draft.pages.shape[1], lens, lens, keep, 2,
                            recent, draft.acc_dev[0], draft.pos_dev[0], draft.acc_dev[0],
                            draft.pos_dev[0], draft.stride, lens_out, room, size))
    assert lens_out.item() == keep
    for p, w in zip(c.pools, want[:2]):
        assert np.array_equal(p.cpu().view(torch.int16).numpy(), w)
    stayed = np.sort(draft.pos_dev[0].cpu().numpy()[0, :, :keep], -1)
    assert (stayed[:, -recent:] == np.arange(length - recent, length)).all()


def test_more_sequences_than_a_launch_takes():
    """66000 trees of three nodes: the root, and two children of which the model chose the second, the
    first or none."""
    n, page, d = 66000, 4, 8
    g = np.random.default_rng(12)
    f = dict(device="cuda")
    pages = g.permutation(n).astype(np.int32)[:, None]
    k, v = (torch.randn(n, 1, page, d, **f) for _ in range(2))
    acc = torch.rand(n, 1, page, **f)
    pos = torch.randint(0, 1 << 30, (n, 1, page), dtype=torch.int32, **f)
    choice = g.integers(5, 8, n)  # children 5 and 6
    tokens = np.tile([4, 5, 6], n).astype(np.int32)
    chosen = np.stack([choice, np.zeros(n), np.full(n, 9)], 1).reshape(-1).astype(np.int32)
    outs = [torch.full((3 * n,), 77, dtype=torch.int32, **f)] + [
        torch.full((n,), 77, dtype=torch.int32, **f) for _ in range(3)]
    wants = []
    second = torch.from_numpy(choice == 6).cuda()
    at = dev(pages[:, 0]).long()
    for t, rows in ((k, at), (v, at), (acc, torch.arange(n, **f)), (pos, torch.arange(n, **f))):
        w = t.clone()
        r = rows[second]
        w[r, :, 2] = t[r, :, 3]  # slot 1 + 2 to slot 1 + 1
        wants.append(w)
    wq.check(wq.wq_kv_accept_slots(
        wq.kv_cache(k, v), n, 3 * n, dev(pages), 1, dev((3 * np.arange(n + 1)).astype(np.int32)),
        dev(np.tile([-1, 0, 0], n).astype(np.int32)), dev(tokens), dev(chosen),
        torch.full((n,), 4, dtype=torch.int32, **f), *outs, wq.slot_arrays([acc], [pos]), page))
    torch.cuda.synchronize()
    for got, want in zip((k, v, acc, pos), wants):
        assert torch.equal(got, want)
    path = np.full((n, 3), -1)
    path[:, 0] = 0
    path[choice == 5, 1], path[choice == 6, 1] = 1, 2
    count = np.where(choice == 7, 1, 2)
    assert (outs[0].cpu().numpy().reshape(n, 3) == path).all()
    assert (outs[1].cpu().numpy() == count).all() and (outs[3].cpu().numpy() == 1 + count).all()
    assert (outs[2].cpu().numpy() == np.choose(choice - 5, [0, 9, 7])).all()
