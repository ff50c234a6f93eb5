"""The library is built and called where the binding's C module cannot be built."""
import os
import sys
import sysconfig

import numpy as np
import pytest

import gemv_transformer_gb300 as wq
from gemv_transformer_gb300 import build as wqbuild
from test_py_calls import NAMES, good


@pytest.fixture
def no_module(monkeypatch, tmp_path):
    """As in a checkout whose Python has no headers."""
    wqbuild.build()
    wq.load()
    built = wq.CALLS_PATH
    monkeypatch.setattr(wqbuild, "CALLS", str(tmp_path / "none.so"))
    monkeypatch.setattr(wqbuild.sysconfig, "get_paths", lambda *a, **k: {"include": str(tmp_path)})
    monkeypatch.setattr(wq, "CALLS_PATH", str(tmp_path / "none.so"))
    monkeypatch.setattr(wq, "_calls", None)
    return built


def test_the_library_does_not_need_the_module(no_module):
    assert wqbuild.up_to_date()
    assert wqbuild.build() == wqbuild.LIB and not os.path.exists(wqbuild.CALLS)


def test_a_module_that_does_not_compile_is_an_error(monkeypatch, tmp_path):
    wqbuild.build()
    src = tmp_path / "bad.c"
    src.write_text("int x = ;\n")
    monkeypatch.setattr(wqbuild, "CALLS", str(tmp_path / "none.so"))
    monkeypatch.setattr(wqbuild, "CALLS_SRC", str(src))
    with pytest.raises(RuntimeError, match="gcc failed"):
        wqbuild.build()
    assert wqbuild._newer(wqbuild.LIB, wqbuild._deps())


@pytest.mark.parametrize("name", NAMES)
def test_calls_go_through_ctypes(no_module, name):
    call = getattr(wq, name)
    assert call(*good(name)) == wq.WQ_ERR_INVALID_ARG
    assert call(*[np.int64(x) if type(x) is int else x for x in good(name)]) == wq.WQ_ERR_INVALID_ARG
    a = good(name)
    a[1] = 2.5
    with pytest.raises(TypeError):
        call(*a)
    a = good(name)
    a[-1] = "x"
    with pytest.raises(AttributeError):
        call(*a)


@pytest.mark.gpu
def test_the_same_results_through_ctypes(no_module):
    import test_attn_paged_gpu as t
    g = np.random.default_rng(1)
    lens = [300, 41]
    c = t.Cache(g, lens, 2, 64, "bf16", 16)
    q = t.queries(g, 2, 4, 64)
    slow = t.check(c, lens, 4, q, 0.125, with_acc=True)
    assert not hasattr(wq._calls, "bind")
    wq._calls, wq.CALLS_PATH = None, no_module
    fast = t.check(c, lens, 4, q, 0.125, with_acc=True)
    assert hasattr(wq._calls, "bind")
    for a, b in zip(slow, fast):
        assert np.array_equal(a, b)


def test_the_module_is_one_interpreter_s():
    """Its name carries the interpreter's tag, and the binding loads that name alone."""
    tag = sysconfig.get_config_var("EXT_SUFFIX")
    assert sys.implementation.cache_tag.split("-")[-1] in tag
    assert os.path.basename(wqbuild.CALLS) == os.path.basename(wq.CALLS_PATH) == "_wq_calls" + tag
