"""Host-side refusals and marshalling of wq_kv_accept_slots (CPU only)."""
import ctypes

import pytest

import gemv_transformer_gb300 as wq
from gemv_transformer_gb300 import build as wqbuild
from test_kv_abi import CACHES, cache
from test_py_calls import Index, Stream, Tensor

A = 0x10000  # a 16-byte aligned fake device address: never dereferenced below
BAD = wq.WQ_ERR_INVALID_ARG


@pytest.fixture(scope="module", autouse=True)
def lib():
    wqbuild.build()
    return wq.load()


def call(c=None, ns=2, n=8, pages=A, wide=4, starts=A, parent=A, tokens=A, choice=A, lens=A,
         path=A, count=A, nxt=A, out=2 * A, slots=((A, A),), stride=64):
    c = c or [cache()]
    if slots is not None:
        slots = (wq.SlotArrays * len(slots))(*[wq.SlotArrays(*x) for x in slots])
    return wq.wq_kv_accept_slots((wq.KvCache * len(c))(*c), ns, n, pages, wide, starts, parent,
                                 tokens, choice, lens, path, count, nxt, out, slots, stride, 0)


@pytest.mark.parametrize("kw", [
    dict(ns=0), dict(n=0), dict(pages=None), dict(wide=0), dict(wide=1 << 27), dict(starts=None),
    dict(parent=None), dict(tokens=None), dict(choice=None), dict(lens=None), dict(path=None),
    dict(count=None), dict(nxt=None), dict(out=None), dict(out=A), dict(slots=None),
    dict(slots=[(A + 2, A)]), dict(slots=[(A, A + 1)]), dict(stride=0), dict(stride=-5),
    dict(c=[cache(), cache(n_heads=1)], slots=[(A, A)] * 2),
    dict(c=[cache(), cache()], slots=[(A, A), (None, A + 2)])] + [dict(c=[cache(**c)]) for c in CACHES])
def test_refusals(kw):
    assert call(**kw) == BAD


def test_arguments():
    t, s = Tensor, Stream()
    good = [cache(), 0, Index(), t(), 4, t(), t(), t(), t(), t(), t(), t(), t(), t(2 * A),
            wq.SlotArrays(A, None), 64, s]
    assert wq.wq_kv_accept_slots(*good) == BAD
    for i, wrong in ((0, "x"), (3, 2.5), (14, (wq.SlotArrays * 2)()), (15, None), (16, "x")):
        a = list(good)
        a[i] = wrong
        with pytest.raises((TypeError, AttributeError, ctypes.ArgumentError)):
            wq.wq_kv_accept_slots(*a)


def test_slot_arrays():
    import torch
    acc, pos = torch.zeros(2, 3, 9), torch.zeros(2, 3, 9, dtype=torch.int32)
    a = wq.slot_arrays([acc, None], [None, pos])
    assert [(x.acc, x.slot_pos) for x in a] == [(acc.data_ptr(), None), (None, pos.data_ptr())]
    with pytest.raises(ValueError):
        wq.slot_arrays([acc], [])
