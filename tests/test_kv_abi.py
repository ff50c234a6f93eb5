"""Host-side refusals of the rotary and paged-cache calls, and workspace sizes (CPU only)."""
import ctypes

import pytest

import gemv_transformer_gb300 as wq
from gemv_transformer_gb300 import build as wqbuild

A = 0x10000  # a 16-byte aligned fake device address: never dereferenced below
BAD = wq.WQ_ERR_INVALID_ARG


@pytest.fixture(scope="module", autouse=True)
def lib():
    wqbuild.build()
    return wq.load()


def cache(**kw):
    base = dict(k=A, v=A, dtype=wq.WQ_BF16, n_pages=10, page_size=16, n_heads=2, head_dim=64,
                reserved=0, page_stride=2048, head_stride=1024, token_stride=64)
    base.update(kw)
    return wq.KvCache(*base.values())


def table(rows=8, rot=64, base=10000.0, scaling=None, out=A):
    return wq.wq_rope_table(rows, rot, base, scaling, out, 0)


def scaling(**kw):
    s = dict(kind=wq.WQ_ROPE_BANDS, original=1024, factor=4.0, low=1.0, high=4.0, magnitude=0.0)
    s.update(kw)
    return wq.RopeScaling(*s.values())


@pytest.mark.parametrize("kw", [
    dict(rows=0), dict(rot=0), dict(rot=63), dict(rot=258), dict(base=1.0), dict(base=float("nan")),
    dict(base=float("inf")), dict(out=None), dict(out=A + 4),
    dict(scaling=scaling(kind=5)), dict(scaling=scaling(kind=-1)), dict(scaling=scaling(factor=0.0)),
    dict(scaling=scaling(factor=float("nan"))), dict(scaling=scaling(original=0)),
    dict(scaling=scaling(low=0.0)), dict(scaling=scaling(low=4.0)),
    dict(scaling=scaling(magnitude=-1.0)), dict(scaling=scaling(magnitude=float("inf"))),
    dict(scaling=scaling(kind=wq.WQ_ROPE_NTK), rot=2)])
def test_rope_table_refusals(kw):
    assert table(**kw) == BAD


def rope(n=2, h=2, d=64, rot=64, flags=0, x=A, xs=128, pos=A, tab=A, rows=8, out=2 * A, os=128):
    return wq.wq_rope(n, h, d, rot, flags, x, xs, pos, tab, rows, out, os, 0)


@pytest.mark.parametrize("kw", [
    dict(n=0), dict(h=0), dict(d=0), dict(d=258, xs=1000, os=1000), dict(rot=-2), dict(rot=7),
    dict(rot=66), dict(flags=4), dict(x=None), dict(out=None), dict(x=A + 2), dict(out=A + 1),
    dict(xs=127), dict(os=127), dict(xs=1 << 30), dict(pos=None), dict(tab=None), dict(tab=A + 8),
    dict(rows=0), dict(out=A, os=132)])
def test_rope_refusals(kw):
    assert rope(**kw) == BAD


CACHES = [dict(k=None), dict(v=None), dict(k=A + 8), dict(v=A + 2), dict(dtype=wq.WQ_Q8_0),
          dict(dtype=9), dict(n_pages=0), dict(page_size=0), dict(n_heads=0), dict(head_dim=0),
          dict(head_dim=60), dict(head_dim=264), dict(page_stride=63), dict(head_stride=1028),
          dict(token_stride=56), dict(token_stride=-64), dict(page_stride=1 << 62)]


def append(c=None, n=2, hq=2, rot=64, flags=0, q=A, qs=256, k=A, ks=256, v=A, vs=256, pos=A, tab=A,
           rows=8, ns=2, seq=None, slot=A, pages=A, wide=4, out=2 * A, os=128, acc=None, sp=None,
           st=0):
    return wq.wq_kv_append(c or cache(), n, hq, rot, flags, q, qs, k, ks, v, vs, pos, tab, rows, ns,
                           seq, slot, pages, wide, out, os, acc, sp, st, 0)


@pytest.mark.parametrize("kw", [
    dict(n=0), dict(hq=-1), dict(rot=3), dict(rot=66), dict(flags=8), dict(q=None), dict(qs=100),
    dict(k=None), dict(k=A + 2), dict(ks=127), dict(v=None), dict(vs=127), dict(pos=None),
    dict(tab=None), dict(rows=0), dict(ns=0), dict(ns=1), dict(slot=None), dict(pages=None),
    dict(wide=0), dict(wide=1 << 27), dict(out=None), dict(os=64), dict(out=A, os=128),
    dict(acc=A), dict(sp=A), dict(sp=A, st=8, pos=None, rot=0)] + [dict(c=cache(**c)) for c in CACHES])
def test_append_refusals(kw):
    assert append(**kw) == BAD


def attn(c=None, n=2, hq=4, scale=0.1, window=0, q=A, qs=256, pages=A, wide=4, lens=A, mask=None,
         ms=0, out=2 * A, os=256, lse=None, ain=None, aout=None, st=0, room=A, size=1 << 30):
    return wq.wq_attn_paged(c or cache(), n, hq, scale, window, q, qs, pages, wide, lens, mask, ms,
                            out, os, lse, ain, aout, st, room, size, 0)


@pytest.mark.parametrize("kw", [
    dict(n=0), dict(hq=0), dict(hq=3), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(window=-1), dict(q=None), dict(q=A + 4), dict(qs=255), dict(qs=258), dict(pages=None),
    dict(wide=0), dict(wide=1 << 27), dict(lens=None), dict(mask=A), dict(out=None),
    dict(out=A + 8), dict(os=252), dict(os=257), dict(ain=A), dict(aout=A), dict(ain=A, st=64)]
    + [dict(c=cache(**c)) for c in CACHES])
def test_attention_refusals(kw):
    assert attn(**kw) == BAD


def evict(c=None, n=2, pages=A, wide=4, lens=A, seen=A, keep=8, sinks=0, recent=0, acc=A, sp=A,
          aout=A, pout=A, st=64, lout=A, room=A, size=1 << 30):
    return wq.wq_kv_evict(c or cache(), n, pages, wide, lens, seen, keep, sinks, recent, acc, sp, aout,
                          pout, st, lout, room, size, 0)


@pytest.mark.parametrize("kw", [
    dict(n=0), dict(pages=None), dict(wide=0), dict(wide=1 << 27), dict(lens=None),
    dict(seen=None), dict(keep=0), dict(sinks=-1), dict(recent=-1), dict(sinks=5, recent=4),
    dict(sinks=1 << 30, recent=(1 << 30) + (1 << 29) + 5), dict(acc=None), dict(sp=None),
    dict(aout=None), dict(pout=None), dict(st=0), dict(lout=None), dict(room=None),
    dict(room=A + 16), dict(size=8)] + [dict(c=cache(**c)) for c in CACHES])
def test_evict_refusals(kw):
    assert evict(**kw) == BAD


def test_workspace_sizes():
    c = cache()
    assert wq.wq_kv_evict_workspace_bytes(c, 2, 4, 8) > 0
    assert wq.wq_kv_evict_workspace_bytes(c, 0, 4, 8) == 0
    assert wq.wq_kv_evict_workspace_bytes(cache(head_dim=60), 2, 4, 8) == 0
    assert wq.wq_attn_paged_workspace_bytes(c, 0, 4, 4, 0) == 0
    assert wq.wq_attn_paged_workspace_bytes(c, 2, 3, 4, 0) == 0
    for with_acc in (0, 1):
        need = wq.wq_attn_paged_workspace_bytes(c, 2, 4, 4, with_acc)
        if need:
            aout = A if with_acc else None
            assert attn(aout=aout, st=64, room=None, size=need) == BAD
            assert attn(aout=aout, st=64, room=A + 16, size=need) == BAD
            assert attn(aout=aout, st=64, size=need - 1) == BAD


def test_the_structs_have_the_header_s_layout():
    assert ctypes.sizeof(wq.KvCache) == 64 and wq.KvCache.page_stride.offset == 40
    assert ctypes.sizeof(wq.RopeScaling) == 40 and wq.RopeScaling.factor.offset == 8
