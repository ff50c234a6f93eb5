"""Host-side refusals of the calls for several new tokens per sequence (CPU only), and the oracle's
own pins."""
import ctypes

import numpy as np
import pytest

import gemv_transformer_gb300 as wq
from gemv_transformer_gb300 import build as wqbuild
from oracle import tokens as ot
from test_kv_abi import CACHES, cache

A = 0x10000  # a 16-byte aligned fake device address: never dereferenced below
BAD = wq.WQ_ERR_INVALID_ARG
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def lib():
    wqbuild.build()
    return wq.load()


def norm(kind=wq.WQ_HEAD_RMS, eps=1e-6, weight=A, bias=None):
    return wq.HeadNorm(kind, eps, weight, bias)


def axes(rot=64, flags=0, n=2, pairs=(16, 16, 0, 0), rows=8, columns=32, pos=A, step=8, table=A):
    return wq.RopeAxes(rot, flags, n, (ctypes.c_int32 * 4)(*pairs), rows, columns, 0, pos, step,
                       table)


NORMS = [dict(kind=3), dict(kind=-1), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF),
         dict(weight=A + 2), dict(bias=A + 1)]
AXES = [dict(rot=-2), dict(rot=63), dict(rot=66), dict(flags=2), dict(flags=16), dict(n=0),
        dict(n=5), dict(pairs=(16, 15, 0, 0)), dict(pairs=(40, -8, 0, 0)), dict(pairs=(32, 1, 0, 0)),
        dict(flags=4, pairs=(8, 24, 0, 0)), dict(rows=0), dict(columns=31), dict(columns=129),
        dict(columns=0), dict(flags=8, columns=15), dict(pos=None), dict(pos=A + 2),
        dict(table=None), dict(table=A + 8), dict(step=-1)]


def rows(n=2, h=2, d=64, nv=None, ax=None, x=A, xs=128, t=wq.WQ_F32, out=2 * A, os=128):
    return wq.wq_norm_rope(n, h, d, nv or norm(), ax or axes(), x, xs, t, out, os, 0)


@pytest.mark.parametrize("kw", [
    dict(n=0), dict(h=0), dict(d=0), dict(d=258, xs=1000, os=1000), dict(x=None), dict(out=None),
    dict(x=A + 2), dict(out=A + 2), dict(t=wq.WQ_F16, out=A + 1), dict(xs=127), dict(os=127),
    dict(xs=1 << 30), dict(t=wq.WQ_Q8_0), dict(t=9), dict(out=A, os=132),
    dict(out=A, t=wq.WQ_BF16)] + [dict(nv=norm(**k)) for k in NORMS]
    + [dict(ax=axes(**k)) for k in AXES])
def test_norm_rope_refusals(kw):
    assert rows(**kw) == BAD


def grad(n=2, h=2, d=64, nv=None, ax=None, x=A, xs=128, g=2 * A, gs=128, gx=3 * A, gxs=128, gw=A,
         gb=None, room=A, size=1 << 30):
    return wq.wq_norm_rope_grad(n, h, d, nv or norm(), ax or axes(), x, xs, g, gs, gx, gxs, gw, gb,
                                room, size, 0)


@pytest.mark.parametrize("kw", [
    dict(n=0), dict(h=-1), dict(d=300), dict(x=None), dict(g=None), dict(gx=None), dict(xs=100),
    dict(gs=100), dict(gxs=100), dict(gx=A, gxs=132), dict(gx=2 * A, gxs=132), dict(gw=A + 2),
    dict(gb=A + 1), dict(room=None), dict(room=A + 16), dict(size=100),
    dict(nv=norm(kind=0))] + [dict(nv=norm(**k)) for k in NORMS] + [dict(ax=axes(**k)) for k in AXES])
def test_grad_refusals(kw):
    assert grad(**kw) == BAD


def test_grad_too_large():
    assert grad(n=1 << 30, h=2, xs=1 << 20, gs=1 << 20, gxs=1 << 20) == wq.WQ_ERR_TOO_LARGE
    assert wq.wq_norm_rope_grad_workspace_bytes(0, 1, 64) == 0
    assert wq.wq_norm_rope_grad_workspace_bytes(1, 1, 64) > 0


def append(c=None, n=2, hq=2, qn=None, kn=None, ax=None, q=A, qs=256, k=A, ks=256, v=A, vs=256, ns=2,
           seq=None, slot=A, pages=A, wide=4, t=wq.WQ_F32, out=2 * A, os=128, acc=None, sp=None,
           st=0):
    return wq.wq_kv_append_norm(c or cache(), n, hq, qn or norm(), kn or norm(), ax or axes(), q, qs,
                                k, ks, v, vs, ns, seq, slot, pages, wide, t, out, os, acc, sp, st, 0)


@pytest.mark.parametrize("kw", [
    dict(n=0), dict(hq=-1), dict(q=None), dict(qs=100), dict(k=None), dict(k=A + 2), dict(ks=127),
    dict(v=None), dict(vs=127), dict(ns=0), dict(ns=1), dict(slot=None), dict(pages=None),
    dict(wide=0), dict(wide=1 << 27), dict(out=None), dict(os=64), dict(t=7), dict(out=A, os=128),
    dict(out=A, os=256, t=wq.WQ_F16), dict(acc=A), dict(sp=A), dict(sp=A, st=8, ax=axes(rot=0))]
    + [dict(c=cache(**c)) for c in CACHES] + [dict(qn=norm(**k)) for k in NORMS]
    + [dict(kn=norm(**k)) for k in NORMS] + [dict(ax=axes(**k)) for k in AXES])
def test_append_refusals(kw):
    assert append(**kw) == BAD


def attn(c=None, ns=2, n=8, hq=4, scale=0.1, form=None, t=wq.WQ_BF16, q=A, qs=256, starts=A,
         pages=A, wide=4, lens=A, ot_=wq.WQ_BF16, out=2 * A, os=256, room=A, size=1 << 40):
    return wq.wq_attn_tokens(c or cache(), ns, n, hq, scale, form, t, q, qs, starts, pages, wide,
                             lens, ot_, out, os, None, room, size, 0)


def form(**kw):
    f = wq.AttnForm()
    for k, v in kw.items():
        setattr(f, k, v)
    return f


@pytest.mark.parametrize("kw", [
    dict(ns=0), dict(n=0), dict(hq=0), dict(hq=3), dict(scale=NAN), dict(scale=INF), dict(t=1),
    dict(t=wq.WQ_F32, ot_=wq.WQ_BF16), dict(ot_=wq.WQ_F16), dict(q=None), dict(q=A + 8),
    dict(qs=255), dict(qs=260), dict(starts=None), dict(pages=None), dict(lens=None),
    dict(out=None), dict(out=A + 8), dict(os=255), dict(os=260), dict(wide=0), dict(wide=1 << 27),
    dict(n=1 << 28, hq=8, qs=512, os=512), dict(room=None), dict(room=A + 16), dict(size=1000),
    dict(form=form(softcap=-1.0)), dict(form=form(softcap=NAN)), dict(form=form(window=-1)),
    dict(form=form(tree=A)), dict(form=form(tree=A, tree_stride=1 << 40)), dict(form=form(tree=A, tree_stride=1, prefix=A)),
    dict(form=form(pos=A))] + [dict(c=cache(**c)) for c in CACHES])
def test_attn_refusals(kw):
    assert attn(**kw) == BAD


def test_attn_workspace():
    size = wq.wq_attn_tokens_workspace_bytes
    assert size(cache(), 2, 8, 4, wq.WQ_BF16) > 0
    assert size(cache(), 0, 8, 4, wq.WQ_BF16) == 0 and size(cache(), 2, 0, 4, wq.WQ_BF16) == 0
    assert size(cache(), 2, 8, 3, wq.WQ_BF16) == 0 and size(cache(), 2, 8, 4, wq.WQ_Q4_0) == 0
    assert size(cache(dtype=9), 2, 8, 4, wq.WQ_F32) == 0


def accept(c=None, nc=1, ns=2, n=8, pages=A, wide=4, starts=A, parent=A, tokens=A, choice=A, lens=A,
           path=A, count=A, nxt=A, out=2 * A):
    c = c or [cache()]
    arr = (wq.KvCache * len(c))(*c)
    return wq.load().wq_kv_accept(arr, nc, ns, n, pages, wide, starts, parent, tokens, choice, lens,
                                  path, count, nxt, out, 0)


@pytest.mark.parametrize("kw", [
    dict(nc=0), dict(ns=0), dict(n=0), dict(pages=None), dict(wide=0), dict(wide=1 << 27),
    dict(starts=None), dict(parent=None), dict(tokens=None), dict(choice=None), dict(lens=None),
    dict(path=None), dict(count=None), dict(nxt=None), dict(out=None), dict(out=A),
    dict(c=[cache(), cache(n_heads=1)], nc=2), dict(c=[cache(), cache(token_stride=72)], nc=2),
    dict(c=[cache(), cache(dtype=wq.WQ_F16)], nc=2), dict(c=[cache(), cache(k=None)], nc=2)]
    + [dict(c=[cache(**c)]) for c in CACHES])
def test_accept_refusals(kw):
    assert accept(**kw) == BAD


def test_pair_maps():
    assert ot.pair_map([2, 1]) == [(0, 0), (0, 1), (1, 2)]
    assert ot.pair_map([2, 1], restart=True) == [(0, 0), (0, 1), (1, 0)]
    assert ot.pair_map([4, 2, 2], dealt=True) == [
        (0, 0), (1, 1), (2, 2), (0, 3), (1, 4), (2, 5), (0, 6), (0, 7)]


def test_oracle_attention_by_hand():
    """Two tokens behind one slot, v = 1, 2, 4 and equal scores."""
    k = np.zeros((1, 1, 4, 2))
    v = np.zeros((1, 1, 4, 2))
    v[0, 0, :3, 0] = 1, 2, 4
    q = np.ones((2, 1, 2))
    r = ot.attention(q, k, v, np.zeros((1, 1), int), [0, 2], [3], 1.0)
    assert np.allclose(r["out"][:, 0, 0], [1.5, 7 / 3]) and np.allclose(r["lse"][:, 0],
                                                                       np.log([2, 3]))
    r = ot.attention(q, k, v, np.zeros((1, 1), int), [0, 2], [3], 1.0, tree=[{0}, {1}])
    assert np.allclose(r["out"][:, 0, 0], [1.5, 2.5])
    r = ot.attention(q, k, v, np.zeros((1, 1), int), [0, 2], [3], 1.0, window=1, prefix=[3])
    assert np.allclose(r["out"][:, 0, 0], [3.0, 4.0])


def test_oracle_accept_by_hand():
    parent = [-1, 0, 0, 1, 2, 4]
    tokens = [9, 5, 5, 7, 7, 3]
    assert ot.accept([0, 6], parent, tokens, [5, 7, 7, 1, 3, 2], [10])[4] == [[0, 1, 3]]
    path, count, nxt, lens, _ = ot.accept([0, 6], parent, tokens, [5, 8, 7, 1, 3, 2], [10])
    assert path.tolist() == [0, 1, -1, -1, -1, -1] and (count[0], nxt[0], lens[0]) == (2, 8, 6)
