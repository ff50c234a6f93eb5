"""wq_kv_accept against the oracle: whole numbers and moved rows, all exact."""
import numpy as np
import pytest
import torch

import gemv_transformer_gb300 as wq
from helpers import dev
from kv_helpers import Cache, bits
from oracle import tokens as ot
from tokens_helpers import random_tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from gemv_transformer_gb300 import build
    build.build()
    wq.load()


class Draft:
    def __init__(self, seed, counts, contexts, layers=1, hkv=2, d=64, kind="bf16", page=16,
                 major="head", agree=0.7, chain=False):
        g = np.random.default_rng(seed)
        self.counts, self.contexts = counts, contexts
        self.starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.lens = np.array([a + b for a, b in zip(counts, contexts)], np.int32)
        parent, tokens, choice = [], [], []
        for c in counts:
            p = list(range(-1, c - 1)) if chain else random_tree(g, c)[0]
            t, ch = g.integers(0, 5, c), g.integers(0, 5, c)
            for j in range(c):  # the model often agrees with a child
                kids = [x for x in range(c) if p[x] == j]
                if kids and g.random() < agree:
                    ch[j] = t[g.choice(kids)]
            parent += p
            tokens += list(t)
            choice += list(ch)
        self.parent, self.tokens, self.choice = (np.array(v, np.int32)
                                                 for v in (parent, tokens, choice))
        self.caches = [Cache(np.random.default_rng(seed + i), self.lens, hkv, d, kind, page, major)
                       for i in range(layers)]
        # One table for all layers.
        first = self.caches[0]
        self.page, self.pages = page, first.pages
        for c in self.caches[1:]:
            for a, b in zip(c.pools, first.pools):
                a.copy_(b.flip(0))

    def run(self, one=False):
        n, m = len(self.counts), max(1, len(self.parent))
        f = dict(device="cuda", dtype=torch.int32)
        self.path = torch.full((m + 3,), 77, **f)
        self.accepted, self.next, self.lens_out = (torch.full((n + 2,), 77, **f) for _ in range(3))
        arr = self.caches[0].desc if one else (wq.KvCache * len(self.caches))(
            *[c.desc for c in self.caches])
        pad = [dev(x) if len(x) else torch.zeros(1, **f)
               for x in (self.parent, self.tokens, self.choice)]
        wq.check(wq.wq_kv_accept(arr, n, m, dev(self.pages), self.pages.shape[1], dev(self.starts),
                                 *pad, dev(self.lens), self.path, self.accepted, self.next,
                                 self.lens_out))
        torch.cuda.synchronize()

    def check(self):
        n = len(self.counts)
        path, count, nxt, lens, nodes = ot.accept(self.starts, self.parent, self.tokens,
                                                  self.choice, self.lens)
        before = [[bits(p).reshape(p.shape[:3] + (-1,)).copy() for p in c.pools]
                  for c in self.caches]
        self.run()
        m = len(self.parent)
        assert self.path.cpu().numpy()[:m].tolist() == path.tolist()
        assert (self.path[max(1, m):] == 77).all()
        for got, want in ((self.accepted, count), (self.next, nxt), (self.lens_out, lens)):
            assert got.cpu().numpy()[:n].tolist() == list(want) and (got[n:] == 77).all()
        for c, pools in zip(self.caches, before):
            for pool, want in zip(c.pools, pools):
                old = want.copy()
                for s in range(n):
                    b = self.lens[s] - self.counts[s]
                    for i, node in enumerate(nodes[s]):
                        src, dst = b + node, b + i
                        want[self.pages[s, dst // self.page], :, dst % self.page] = \
                            old[self.pages[s, src // self.page], :, src % self.page]
                assert (bits(pool).reshape(want.shape) == want).all()
        assert wq.wq_get_device_status() == wq.WQ_OK
        return count


@pytest.mark.parametrize("kind,page,major", [("bf16", 16, "head"), ("f16", 7, "token"),
                                             ("f32", 1, "gap"), ("bf16", 100, "head")])
@pytest.mark.parametrize("counts,contexts", [
    ([1], [0]), ([2], [5]), ([16], [100]), ([32, 0, 33, 1, 64], [0, 9, 31, 4, 100]),
    ([130, 7], [3, 50]), ([31, 65, 97], [1, 1, 1])])
def test_accept(kind, page, major, counts, contexts):
    d = Draft(1, counts, contexts, 2, 3, 40, kind, page, major)
    d.check()


@pytest.mark.parametrize("chain", [False, True])
@pytest.mark.parametrize("agree", [0.0, 1.0])
def test_none_and_all(agree, chain):
    d = Draft(2, [40, 100, 33], [7, 20, 0], 3, 2, 128, agree=agree, chain=chain)
    count = d.check()
    if chain and agree:
        assert count.tolist() == [40, 100, 33]


def test_many_layers_and_sequences():
    g = np.random.default_rng(3)
    counts = [int(x) for x in g.integers(0, 6, 300)]
    Draft(3, counts, [int(x) for x in g.integers(0, 9, 300)], 2, 1, 8, "f32", 4).check()
    Draft(4, [9, 20], [10, 3], 53, 1, 16).check()  # more layers than one launch takes


def test_twice_the_same_bits_and_captured():
    """Replayed on the moved cache the call moves the same slots again."""
    a, b = (Draft(5, [24, 50], [30, 8], 2) for _ in range(2))
    a.run(), a.run()
    torch.cuda.synchronize()
    f = dict(device="cuda", dtype=torch.int32)
    outs = [torch.zeros(74, **f)] + [torch.zeros(2, **f) for _ in range(3)]
    arr = (wq.KvCache * 2)(*[c.desc for c in b.caches])
    ins = [dev(x) for x in (b.pages, b.starts, b.parent, b.tokens, b.choice, b.lens)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wq.check(wq.wq_kv_accept(arr, 2, 74, ins[0], b.pages.shape[1], *ins[1:], *outs))
    graph.replay(), graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(a.caches, b.caches):
        for p, q in zip(x.pools, y.pools):
            assert (bits(p) == bits(q)).all()


def test_bad_indexes():
    d = Draft(6, [20, 30, 10, 5], [40, 12, 3, 2])
    d.starts = np.array([0, 20, 15, 60, 65], np.int32)  # sequence 1 falls
    d.lens[2] = 10 ** 6
    d.lens[3] = 4
    want = bits(d.caches[0].pools[0]).copy()
    d.run(one=True)
    assert wq.wq_get_device_status() == wq.WQ_ERR_BAD_INDEX
    assert d.accepted.tolist()[1:4] == [0, 0, 0] and d.next.tolist()[1:4] == [-1, -1, -1]
    assert d.lens_out.tolist()[1:4] == [42, 10 ** 6, 4]
    assert (d.path[20:] == 77).all()
    got = bits(d.caches[0].pools[0])
    assert got.shape == want.shape
    # A page out of range: its nodes stay, the others move.
    d = Draft(7, [40], [40], agree=1.0, chain=False, page=8)
    d.pages = d.pages.copy()
    d.pages[0, 6] = 10 ** 6
    d.run()
    assert wq.wq_get_device_status() == wq.WQ_ERR_BAD_INDEX
    assert d.accepted[0] > 1
