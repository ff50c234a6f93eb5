"""Arguments of the calls for several new tokens per sequence, through the C module and through
ctypes: wrong types and sizes raise their own errors (CPU only; no call gets as far as a launch)."""
import ctypes

import numpy as np
import pytest

import gemv_transformer_gb300 as wq
from gemv_transformer_gb300 import build as wqbuild
from test_calls_build import no_module  # noqa: F401
from test_py_calls import A, Index, LikeCache, Stream, Tensor, cache

NAMES = ["wq_norm_rope", "wq_norm_rope_grad", "wq_kv_append_norm", "wq_attn_tokens", "wq_kv_accept"]
# Strides and byte counts are 64-bit, the other integers C ints.
WIDE = {"wq_norm_rope": (6, 9), "wq_norm_rope_grad": (6, 8, 10, 14),
        "wq_kv_append_norm": (7, 9, 11, 19, 22), "wq_attn_tokens": (8, 15, 18), "wq_kv_accept": ()}


@pytest.fixture(scope="module", autouse=True)
def lib():
    wqbuild.build()
    return wq.load()


def norm():
    return wq.HeadNorm(wq.WQ_HEAD_RMS, 1e-6, A, None)


def axes():
    return wq.RopeAxes(64, 0, 2, (ctypes.c_int32 * 4)(16, 16, 0, 0), 8, 32, 0, A, 8, A)


def good(name):
    """Arguments that are refused late (INVALID_ARG), each pointer an object, the stream one too."""
    t, s = Tensor, Stream()
    if name == "wq_norm_rope":
        return [0, 2, 64, norm(), axes(), t(), 128, wq.WQ_F32, t(2 * A), 128, s]
    if name == "wq_norm_rope_grad":
        return [0, 2, 64, norm(), axes(), t(), 128, t(2 * A), 128, t(3 * A), 128, t(), t(), t(),
                1 << 30, s]
    if name == "wq_kv_append_norm":
        return [cache(), 0, 2, norm(), norm(), axes(), t(), 256, t(), 256, t(), 256, 2, None, t(), t(),
                4, wq.WQ_F32, t(2 * A), 128, None, None, 0, s]
    if name == "wq_attn_tokens":
        return [cache(), 0, 8, 4, 0.1, wq.AttnForm(), wq.WQ_F32, t(), 256, t(), t(), 4, t(),
                wq.WQ_F32, t(2 * A), 256, None, t(), 1 << 30, s]
    return [(wq.KvCache * 2)(cache(), cache()), 0, 8, t(), 4, t(), t(), t(), t(), t(), t(), t(),
            t(), t(2 * A), s]


@pytest.mark.parametrize("name", NAMES)
def test_good_types_reach_the_call(name):
    assert getattr(wq, name)(*good(name)) == wq.WQ_ERR_INVALID_ARG
    a = [Index() if x == 64 and type(x) is int else np.int64(x) if type(x) is int else x
         for x in good(name)]
    assert getattr(wq, name)(*a) == wq.WQ_ERR_INVALID_ARG


@pytest.mark.parametrize("name", NAMES)
def test_a_wrong_argument_raises_its_own_error(name):
    for i, x in enumerate(good(name)):
        wrong = []
        if type(x) is int:
            wrong += [("x", TypeError), (2.5, TypeError), (None, TypeError), (1 << 70, OverflowError)]
            if i not in WIDE[name]:
                wrong.append((1 << 40, OverflowError))
        elif type(x) is float:
            wrong += [("x", TypeError), (None, TypeError)]
        elif isinstance(x, Tensor):
            wrong += [("x", AttributeError), (2.5, AttributeError)]
        elif isinstance(x, Stream):
            wrong += [("x", AttributeError), (2.5, AttributeError)]
        else:  # a descriptor, or the array of caches
            if x is None:
                continue
            wrong += [(v, TypeError) for v in ("x", 5, bytes(80), LikeCache(), wq.RopeScaling(),
                                               (ctypes.c_int64 * 18)())]
        for value, error in wrong:
            a = good(name)
            a[i] = value
            with pytest.raises(error):
                getattr(wq, name)(*a)


@pytest.mark.parametrize("name", NAMES)
def test_counts_of_arguments(name):
    a = good(name)
    for wrong in (a[:4], a + [0, 0], []):
        with pytest.raises(TypeError):
            getattr(wq, name)(*wrong)


def test_descriptors_may_be_missing():
    for name, at in (("wq_norm_rope", (3, 4)), ("wq_norm_rope_grad", (4,)),
                     ("wq_kv_append_norm", (3, 4, 5)), ("wq_attn_tokens", (5,))):
        a = good(name)
        for i in at:
            a[i] = None
        assert getattr(wq, name)(*a) == wq.WQ_ERR_INVALID_ARG


def test_one_cache_or_an_array():
    a = good("wq_kv_accept")
    a[0] = cache()
    assert wq.wq_kv_accept(*a) == wq.WQ_ERR_INVALID_ARG


@pytest.mark.parametrize("name", NAMES)
def test_through_ctypes(no_module, name):  # noqa: F811
    call = getattr(wq, name)
    assert call(*good(name)) == wq.WQ_ERR_INVALID_ARG
    assert call(*[np.int64(x) if type(x) is int else x for x in good(name)]) == wq.WQ_ERR_INVALID_ARG
    a = good(name)
    a[-1] = "x"
    with pytest.raises(AttributeError):
        call(*a)


class Pool:
    """A view of [page][head][row][dim] as far as a descriptor asks."""

    def __init__(self, at, shape=(4, 2, 8, 64)):
        import torch
        self.t = torch.empty(shape, dtype=torch.bfloat16, device="meta")
        self.at = at

    def __getattr__(self, name):
        return getattr(self.t, name)

    def data_ptr(self):
        return self.at


def test_descriptor_helpers():
    import torch
    c = wq.kv_caches([Pool(A), Pool(2 * A)], [Pool(3 * A), Pool(4 * A)])
    assert [(x.k, x.v, x.n_pages, x.page_size) for x in c] == [(A, 3 * A, 4, 8), (2 * A, 4 * A, 4, 8)]
    with pytest.raises(ValueError):
        wq.kv_caches([Pool(A)], [])
    pos = torch.zeros(2, 9, dtype=torch.int32)
    table = torch.zeros(7, 32, 2)
    r = wq.rope_axes(64, 0, [16, 16], pos, table)
    assert (r.axes, r.table_rows, r.table_pairs, r.pos_stride) == (2, 7, 32, 9)
    assert list(r.pairs) == [16, 16, 0, 0]
    with pytest.raises(ValueError):
        wq.rope_axes(64, 0, [], pos, table)
    tree = torch.zeros(5, 3, dtype=torch.int32)
    f = wq.attn_form(2.0, 7, tree=tree)
    assert (f.softcap, f.window, f.tree, f.tree_stride, f.pos) == (2.0, 7, tree.data_ptr(), 3, None)
