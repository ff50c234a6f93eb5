"""Arguments of the calls that the C module marshals: wrong types and sizes raise what ctypes
would, whatever the other arguments are (CPU only; no call gets as far as a launch)."""
import ctypes

import numpy as np
import pytest

import gemv_transformer_gb300 as wq
from gemv_transformer_gb300 import build as wqbuild

A = 0x10000


@pytest.fixture(scope="module", autouse=True)
def lib():
    wqbuild.build()
    return wq.load()


class Tensor:
    """An object with data_ptr(), as a tensor is."""

    def __init__(self, at=A):
        self.at, self.asked = at, 0

    def data_ptr(self):
        self.asked += 1
        return self.at


class Index:
    def __index__(self):
        return 64


class Stream:
    cuda_stream = 0


def cache():
    return wq.KvCache(A, A, wq.WQ_BF16, 10, 16, 2, 64, 0, 2048, 1024, 64)


def good(name):
    """Arguments that are refused late (INVALID_ARG), each pointer an object, the stream one too."""
    t, s = Tensor, Stream()
    if name == "wq_rope":
        return [0, 2, 64, 64, 0, t(), 128, t(), t(), 8, t(2 * A), 128, s]
    if name == "wq_kv_append":
        return [cache(), 0, 2, 64, 0, t(), 256, t(), 256, t(), 256, t(), t(), 8, 2, None, t(), t(), 4,
                t(2 * A), 128, None, None, 0, s]
    if name == "wq_attn_paged":
        return [cache(), 0, 4, 0.1, 0, t(), 256, t(), 4, t(), None, 0, t(2 * A), 256, None, None, None,
                0, t(), 1 << 30, s]
    return [cache(), 0, t(), 4, t(), t(), 8, 0, 0, t(), t(), t(), t(), 64, t(), t(), 1 << 30, s]


NAMES = ["wq_rope", "wq_kv_append", "wq_attn_paged", "wq_kv_evict"]


@pytest.mark.parametrize("name", NAMES)
def test_good_types_reach_the_call(name):
    assert getattr(wq, name)(*good(name)) == wq.WQ_ERR_INVALID_ARG


@pytest.mark.parametrize("name", NAMES)
def test_integers_of_other_types(name):
    a = [Index() if x == 64 and type(x) is int else np.int64(x) if type(x) is int else x
         for x in good(name)]
    assert getattr(wq, name)(*a) == wq.WQ_ERR_INVALID_ARG


@pytest.mark.parametrize("name", NAMES)
def test_a_wrong_argument_raises_its_own_error(name):
    """Each argument in turn; what comes after it is objects whose conversion runs Python."""
    for i, x in enumerate(good(name)):
        wrong = []
        if type(x) is int:
            wrong += [("x", TypeError), (2.5, TypeError), (None, TypeError), (1 << 70, OverflowError)]
            if x < 1 << 20 and x not in (64, 128, 256):
                # Strides and sizes are 64-bit, the others C ints.
                wide = {"wq_kv_append": (23,), "wq_attn_paged": (11, 17)}.get(name, ())
                if i not in wide:
                    wrong.append((1 << 40, OverflowError))
        elif type(x) is float:
            wrong += [("x", TypeError), (None, TypeError)]
        elif isinstance(x, Tensor):
            wrong += [("x", AttributeError), (2.5, AttributeError)]
        elif isinstance(x, Stream):
            wrong += [("x", AttributeError), (2.5, AttributeError)]
        for value, error in wrong:
            a = good(name)
            a[i] = value
            with pytest.raises(error):
                getattr(wq, name)(*a)


@pytest.mark.parametrize("name", NAMES)
def test_two_wrong_arguments_raise_the_first_s_error(name):
    a = good(name)
    at = [i for i, x in enumerate(a) if type(x) is int]
    a[at[0]], a[at[-1]] = "x", 1 << 70
    with pytest.raises(TypeError):
        getattr(wq, name)(*a)


def test_nothing_is_asked_after_an_error():
    a = good("wq_rope")
    a[0] = "x"
    with pytest.raises(TypeError):
        wq.wq_rope(*a)
    assert all(x.asked == 0 for x in a if isinstance(x, Tensor))


class LikeCache(ctypes.Structure):
    """The bytes of a KvCache under another name."""
    _fields_ = wq.KvCache._fields_


class SubCache(wq.KvCache):
    pass


@pytest.mark.parametrize("name", NAMES[1:])
def test_only_a_cache_is_a_cache(name):
    for wrong in (bytes(64), bytearray(64), np.zeros(8), (ctypes.c_int64 * 8)(), LikeCache(),
                  bytearray(63), "x", 5, wq.RopeScaling()):
        a = good(name)
        a[0] = wrong
        with pytest.raises(TypeError):
            getattr(wq, name)(*a)
    a = good(name)
    a[0] = SubCache.from_buffer_copy(cache())
    assert getattr(wq, name)(*a) == wq.WQ_ERR_INVALID_ARG
    a[0] = None
    assert getattr(wq, name)(*a) == wq.WQ_ERR_INVALID_ARG
