"""GPU parity of wq_attn_tokens against the f64 oracle.

Tolerances.  With u = 2^-24: a score is a sum of head_dim products, within (head_dim + 8) u of
sx = scale sum |q k| (f32 sums, rounded or cut), plus 8 u of |x| for scale, cap and bias (the fast
tanh of 16-bit queries: 2^-21 of the cap); e_x is that sum, and a weight is within 2 e_x + 16 u of
itself (its maximum and its exponential), its sum over n slots within n u more.  So out is within
(2 e_x + (n + 80) u) of pv = sum p |v|, and lse within e_x + (n + 16) u + 4 u |lse|.  16-bit queries
on the tensor cores round p to their type (half a step of p; f16 also 2^-25 absolute, against the
largest weight of 1 before the division), and out to the out type."""
import numpy as np
import pytest
import torch

import gemv_transformer_gb300 as wq
from helpers import dev, status_ok
from kv_helpers import Cache, workspace
from oracle import tokens as ot
from tokens_helpers import HALF, KINDS, TORCH, as_type, random_tree, tree_words

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    from gemv_transformer_gb300 import build
    build.build()
    wq.load()
    yield
    status_ok()


class Case:
    """New tokens `counts` behind `contexts` slots, and what they see."""

    def __init__(self, seed, counts, contexts, hq, hkv, d, kind="bf16", qtype="bf16", page=16,
                 major="head", tree=False, softcap=0.0, window=0, slopes=False, first=False,
                 prefix=False, own_pos=False, otype=None, scale=None, pad=0, extra=0, qscale=1.0,
                 max_pages=None, fill=np.nan):
        g = np.random.default_rng(seed)
        self.counts, self.hq, self.hkv, self.d, self.kind = counts, hq, hkv, d, kind
        self.qtype, self.otype = qtype, otype or qtype
        self.lens = [a + b for a, b in zip(counts, contexts)]
        self.cache = Cache(g, self.lens, hkv, d, kind, page, major, max_pages, fill=fill)
        self.starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.m = int(self.starts[-1])
        self.rows = self.m + extra  # rows behind the last sequence
        self.stride = hq * d + pad
        self.q, self.q64 = as_type(qscale * g.standard_normal((max(1, self.rows), self.stride)),
                                   qtype)
        self.scale = d ** -0.5 if scale is None else scale
        self.softcap, self.window = softcap, window
        self.slopes = (2.0 ** (-8 * (1 + np.arange(hq)) / hq)).astype(np.float32) if slopes \
            else None
        self.first = self.prefix = self.tree = self.pos = None
        slot = np.concatenate([np.arange(c) + b for c, b in zip(counts, contexts)] + [[]]) \
            .astype(np.int32)
        if first:
            self.first = np.maximum(0, slot - g.integers(0, 40, self.m)).astype(np.int32)
            if self.m > 2:
                self.first[1] = 1 << 30  # sees nothing
        if prefix:
            self.prefix = g.integers(0, 60, len(counts)).astype(np.int32)
        if tree:
            self.tree, pos = [], []
            for c, b in zip(counts, contexts):
                _, above = random_tree(g, c)
                self.tree += above
                pos += [b + len(a) - 1 for a in above]
            if self.m > 3:
                self.tree[2] = set()  # a row without bits
            self.words = max(1, -(-max(counts) // 32)) + 1
            if own_pos:
                self.pos = np.array(pos, np.int32)

    def run(self, out=None, lse=None, stream=None, room=None):
        t = dict(slopes=self.slopes, first=self.first, prefix=self.prefix, pos=self.pos)
        t = {k: None if v is None else dev(v) for k, v in t.items()}
        t["tree"] = None if self.tree is None else tree_words(self.tree, self.words)
        self.keep = t
        form = wq.attn_form(self.softcap, self.window, **t)
        n = len(self.counts)
        rows = max(1, self.rows)
        self.out = torch.full((rows, self.stride), 9.0, device="cuda", dtype=TORCH[self.otype]) \
            if out is None else out
        self.lse = torch.full((rows, self.hq), 9.0, device="cuda") if lse is None else lse
        size = wq.wq_attn_tokens_workspace_bytes(self.cache.desc, n, rows, self.hq,
                                                 KINDS[self.qtype])
        assert size > 0
        self.room = workspace(size) if room is None else room
        self.starts_dev, self.lens_dev = dev(self.starts), dev(np.array(self.lens, np.int32))
        wq.check(wq.wq_attn_tokens(
            self.cache.desc, n, rows, self.hq, self.scale, form, KINDS[self.qtype], self.q,
            self.stride, self.starts_dev, self.cache.pages_dev, self.cache.max_pages,
            self.lens_dev, KINDS[self.otype], self.out, self.stride, self.lse, self.room, size,
            stream), "wq_attn_tokens")
        return self

    def want(self, k=None, v=None):
        hk, hv = self.cache.host()
        q = self.q64[:self.m, :self.hq * self.d].reshape(self.m, self.hq, self.d)
        return ot.attention(q, hk if k is None else k, hv if v is None else v, self.cache.pages,
                            self.starts, self.lens, self.scale, self.softcap, self.window,
                            self.slopes, self.first, self.prefix, self.tree, self.pos)

    def check(self, want=None, rows=None):
        w = want or self.want()
        got = self.out.double().cpu().numpy()
        lse = self.lse.double().cpu().numpy()
        assert (got[self.m:] == 9).all() and (lse[self.m:] == 9).all()
        assert (got[:, self.hq * self.d:] == 9).all()
        got = got[:self.m, :self.hq * self.d].reshape(self.m, self.hq, self.d)
        lse = lse[:self.m]
        tensor = self.qtype != "f32" and self.qtype == self.kind
        n = w["n"][:, None]
        ex = (self.d + 8) * U * w["sx"] + 8 * U * w["mx"]
        if self.softcap:
            ex = ex + 2.0 ** -21 * self.softcap
        rel = 2 * ex + (n + 80) * U
        tol = rel[..., None] * w["pv"]
        if tensor:
            tol = tol + HALF[self.qtype] * w["pv"]
            if self.qtype == "f16":
                tol = tol + 2.0 ** -25 * n[..., None] * np.nanmax(np.abs(w["pv"]), -1,
                                                                 keepdims=True) * 8
        if self.otype != "f32":
            tol = tol + HALF[self.otype] * (np.abs(w["out"]) + tol)
            if self.otype == "f16":
                tol = tol + 2.0 ** -25
        tol_lse = ex + (n + 16) * U + 4 * U * np.abs(np.where(np.isfinite(w["lse"]), w["lse"], 0))
        take = slice(None) if rows is None else rows
        bad = ~(np.abs(got - w["out"]) <= tol)[take]
        assert not bad.any(), (np.argwhere(bad)[:5], np.abs(got - w["out"])[take][bad][:5],
                               tol[take][bad][:5], got[take][bad][:5], w["out"][take][bad][:5])
        none = np.isneginf(w["lse"])
        assert (np.isneginf(lse) == none)[take].all()
        with np.errstate(invalid="ignore"):
            assert (none | (np.abs(lse - w["lse"]) <= tol_lse))[take].all()
        return w


TYPES = [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f32", "f32"), ("f16", "f32"),
         ("f16", "bf16")]


@pytest.mark.parametrize("kind,qtype", TYPES)
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (8, 1, 128), (3, 3, 96), (10, 2, 80), (2, 1, 256),
                                      (16, 1, 40)])
def test_causal(kind, qtype, hq, hkv, d):
    Case(1, [1, 70, 0, 17, 130], [0, 3, 9, 200, 100], hq, hkv, d, kind, qtype).run().check()


@pytest.mark.parametrize("kind,qtype", TYPES)
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (8, 1, 128), (5, 5, 72), (4, 1, 192)])
@pytest.mark.parametrize("own_pos,window", [(False, 0), (True, 30), (False, 20), (True, 0)])
def test_tree(kind, qtype, hq, hkv, d, own_pos, window):
    Case(2, [5, 1, 33, 70], [0, 300, 129, 61], hq, hkv, d, kind, qtype, tree=True, own_pos=own_pos,
         window=window, slopes=own_pos).run().check()


@pytest.mark.parametrize("kind,qtype", TYPES)
@pytest.mark.parametrize("form", [
    dict(softcap=2.0), dict(window=1), dict(window=50), dict(slopes=True), dict(first=True),
    dict(prefix=True), dict(prefix=True, first=True, window=33, softcap=5.0, slopes=True),
    dict(scale=-0.2), dict(scale=0.0), dict(tree=True, first=True, softcap=3.0)],
    ids=lambda f: "-".join(f))
def test_forms(kind, qtype, form):
    Case(3, [40, 3, 90], [20, 150, 0], 8, 2, 128, kind, qtype, **form).run().check()
    Case(4, [40, 3, 90], [20, 150, 0], 2, 2, 64, kind, qtype, **form).run().check()


@pytest.mark.parametrize("kind,qtype", TYPES)
@pytest.mark.parametrize("page,major", [(1, "head"), (7, "token"), (8, "gap"), (24, "head"),
                                        (64, "token"), (100, "gap"), (256, "head")])
def test_pages(kind, qtype, page, major):
    Case(5, [20, 35], [210, 91], 4, 2, 128, kind, qtype, page, major).run().check()
    Case(6, [20, 35], [210, 91], 4, 2, 88, kind, qtype, page, major, tree=True).run().check()


@pytest.mark.parametrize("kind,qtype", TYPES)
@pytest.mark.parametrize("count,context", [(1, 0), (1, 1), (2, 126), (1, 128), (64, 64), (65, 63),
                                           (128, 128), (129, 1), (31, 33), (16, 0), (257, 130)])
def test_edges(kind, qtype, count, context):
    Case(7, [count], [context], 4, 2, 64, kind, qtype).run().check()
    Case(8, [count], [context], 7, 1, 128, kind, qtype).run().check()


@pytest.mark.parametrize("kind,qtype", TYPES)
def test_many_sequences(kind, qtype):
    """More sequences than the plan takes at a time, most of one token, some of none."""
    g = np.random.default_rng(9)
    counts = [int(x) for x in g.choice([0, 1, 1, 1, 2, 5], 1100)]
    contexts = [int(x) for x in g.choice([0, 1, 7, 20], 1100)]
    Case(9, counts, contexts, 2, 1, 64, kind, qtype, page=8).run().check()


@pytest.mark.parametrize("kind,qtype", TYPES)
def test_long_context_split_over_the_grid(kind, qtype):
    Case(10, [3, 20], [5000, 2300], 4, 1, 64, kind, qtype, tree=True).run().check()


@pytest.mark.parametrize("kind,qtype", TYPES)
def test_out_types_strides_and_rows_behind(kind, qtype):
    Case(11, [20, 9], [30, 0], 4, 2, 64, kind, qtype, otype="f32", pad=16, extra=7).run().check()
    Case(12, [150, 0], [30, 0], 4, 2, 128, kind, qtype, pad=8, extra=140).run().check()


@pytest.mark.parametrize("kind,qtype", TYPES)
def test_large_scores(kind, qtype):
    """Weights of one slot, and scores of hundreds."""
    Case(13, [30, 100], [60, 10], 4, 2, 64, kind, qtype, qscale=60.0).run().check()


@pytest.mark.parametrize("kind,qtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("tree", [False, True])
def test_values_that_are_not_finite(kind, qtype, d, value, tree):
    """k and v of some new slots and one old slot are not finite: tokens that do not see them have
    the results without them, tokens that see one have not finite ones in the dims of a bad v and
    everywhere for a NaN in k."""
    counts, contexts = [40, 150], [33, 100]
    c = Case(14, counts, contexts, 4, 2, d, kind, qtype, tree=tree, first=True)
    bad_v, bad_k = [(0, 33 + 20), (1, 100 + 90), (1, 50)], [(0, 33 + 30), (1, 100 + 120)]
    k, v = c.cache.host()
    for pool, bad, host in ((0, bad_k, k), (1, bad_v, v)):
        for s, j in bad:
            p, r = c.cache.pages[s, j // 16], j % 16
            c.cache.pools[pool][p, :, r, 5] = value
            host[p, :, r] = 0
    c.run()
    w = c.want(k, v)
    see = np.zeros((2, c.m), bool)
    for s in range(2):
        for t in range(c.starts[s], c.starts[s + 1]):
            for i, bad in enumerate((bad_k, bad_v)):
                for bs, j in bad:
                    see[i, t] |= bs == s and ot.sees(
                        t - c.starts[s], j, contexts[s], counts[s], c.lens[s], c.first[t],
                        bits=None if not tree else c.tree[t])
    clean = ~see.any(0)
    assert clean.any() and see[1].any()
    c.check(w, clean)
    got = c.out.double().cpu().numpy()[:c.m, :4 * d].reshape(c.m, 4, d)
    only_v = see[1] & ~see[0]
    assert (~np.isfinite(got[only_v][:, :, 5])).all()
    other = np.delete(got[only_v], 5, -1)
    assert np.isfinite(other).all()
    if np.isnan(value):
        assert np.isnan(got[see[0]]).all()


@pytest.mark.parametrize("kind,qtype", TYPES)
def test_bad_indexes(kind, qtype):
    """Pages, lengths and starts out of range leave what they say out and are recorded."""
    c = Case(15, [20, 30, 10], [100, 40, 30], 4, 2, 64, kind, qtype)
    c.cache.pages[1, 1] = -5          # slots 16..31 of sequence 1
    c.cache.pages[0, 2] = 10 ** 6     # slots 32..47 of sequence 0
    c.cache.pages_dev = dev(c.cache.pages)
    c.run()
    assert wq.wq_get_device_status() == wq.WQ_ERR_BAD_INDEX
    c.check()
    # A length above the table's slots is cut, one below the new tokens leaves the first of them
    # with nothing.
    c = Case(16, [20, 30], [100, 40], 4, 2, 64, kind, qtype)
    slots = c.cache.max_pages * 16
    full = c.cache.pages.copy()
    full[full < 0] = c.cache.pages.max()
    c.cache.pages, c.cache.pages_dev = full, dev(full)
    c.cache.pools[0].nan_to_num_(0.25), c.cache.pools[1].nan_to_num_(0.5)
    c.lens = [slots + 50, 12]
    c.run()
    assert wq.wq_get_device_status() == wq.WQ_ERR_BAD_INDEX
    w = c.want()
    assert (w["n"][20:38] == 0).all() and (w["n"][38:] > 0).all()
    c.check(w)
    # A range of tokens that falls or passes n_tok.
    c = Case(17, [20, 30, 10], [10, 4, 3], 4, 2, 64, kind, qtype)
    c.starts = np.array([0, 20, 15, 1000], np.int32)
    c.run()
    assert wq.wq_get_device_status() == wq.WQ_ERR_BAD_INDEX
    assert (c.out[20:].double() == 9).all() and (c.lse[20:] == 9).all()
    assert torch.isfinite(c.out[:20].double()).all() and not (c.out[:20].double() == 9).any()


def test_pool_beyond_four_gigabytes():
    """The last pages of a pool whose offsets pass 2^32 bytes."""
    d, page = 128, 64
    pages = (1 << 32) // (page * d * 2) + 40
    k = torch.empty(pages, 1, page, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    c = Case(18, [30], [226], 4, 1, d, page=page)
    ids = pages - 1 - np.arange(4)
    for pool, big in zip(c.cache.pools, (k, v)):
        for i, p in enumerate(ids):
            big[int(p)] = pool[int(c.cache.pages[0, i])]
    host = c.want()
    c.cache.pages_dev = dev(ids[None].astype(np.int32))
    c.cache.desc, c.cache.max_pages = wq.kv_cache(k, v), 4
    c.run()
    c.check(host)


@pytest.mark.parametrize("kind,qtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_repeated_bits_and_captured_replay(kind, qtype):
    """The same bits again, in a captured graph, on another stream, and beside another call."""
    c = Case(19, [50, 200], [700, 30], 8, 2, 128, kind, qtype).run()
    first = c.out.clone(), c.lse.clone()
    c.run()
    assert torch.equal(first[0], c.out) and torch.equal(first[1], c.lse)
    room, out, lse = c.room, torch.zeros_like(c.out), torch.zeros_like(c.lse)
    out.fill_(9), lse.fill_(9)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        c.run(out, lse, None, room)
    torch.cuda.synchronize()
    out.fill_(9), lse.fill_(9)
    graph = torch.cuda.CUDAGraph()
    other = Case(20, [64], [500], 8, 2, 128, kind, qtype).run()
    with torch.cuda.graph(graph):
        st = torch.cuda.current_stream().cuda_stream
        n = len(c.counts)
        form = wq.attn_form(c.softcap, c.window)
        for _ in range(2):
            wq.check(wq.wq_attn_tokens(
                c.cache.desc, n, c.rows, c.hq, c.scale, form, KINDS[qtype], c.q, c.stride,
                c.starts_dev, c.cache.pages_dev, c.cache.max_pages, c.lens_dev, KINDS[qtype], out,
                c.stride, lse, room, room.numel(), st))
    for _ in range(3):
        graph.replay()
        other.run()
    torch.cuda.synchronize()
    assert torch.equal(first[0], out) and torch.equal(first[1], lse)
    other.check()


def test_a_decode_token_agrees_with_wq_attn_paged():
    """One token per sequence: both calls within their tolerances of one another."""
    c = Case(21, [1, 1, 1], [40, 0, 900], 8, 2, 128, "bf16", "f32").run()
    out = torch.zeros(3, 8 * 128, device="cuda")
    lse = torch.zeros(3, 8, device="cuda")
    size = wq.wq_attn_paged_workspace_bytes(c.cache.desc, 3, 8, c.cache.max_pages, False)
    room = workspace(size)
    wq.check(wq.wq_attn_paged(c.cache.desc, 3, 8, c.scale, 0, c.q, 1024, c.cache.pages_dev,
                              c.cache.max_pages, c.lens_dev, None, 0, out, 1024, lse, None, None, 0,
                              room, size))
    w = c.check()
    pv = w["pv"].reshape(3, -1)
    rel = 4 * (136 * U * w["sx"].max() + 8 * U * w["mx"].max()) + 2 * (901 + 80) * U
    assert (np.abs(out.double().cpu().numpy() - c.out.double().cpu().numpy()) <= rel * pv).all()
