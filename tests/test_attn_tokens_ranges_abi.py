"""Scales and caps of wq_attn_tokens that f32 arithmetic does not hold are refused (CPU only): their
quotient, or their product with log2 e, may be infinite, and 0 times it is NaN."""
import pytest

import gemv_transformer_gb300 as wq
from gemv_transformer_gb300 import build as wqbuild
from test_tokens_abi import attn, form

BAD = wq.WQ_ERR_INVALID_ARG


@pytest.fixture(scope="module", autouse=True)
def lib():
    wqbuild.build()
    return wq.load()


@pytest.mark.parametrize("kw", [
    dict(scale=2.0 ** 61), dict(scale=-3e38), dict(form=form(softcap=1e-39)),
    dict(form=form(softcap=2.0 ** -61)), dict(form=form(softcap=2.0 ** 61)),
    dict(form=form(softcap=3e38)), dict(scale=1e30, form=form(softcap=1e-30))])
def test_refused(kw):
    assert attn(**kw) == BAD

