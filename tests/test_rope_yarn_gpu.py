"""The default magnitude of a YaRN table: 0.1 ln(factor) + 1 above a factor of 1, else 1."""
import math

import numpy as np
import pytest
import torch

import gemv_transformer_gb300 as wq
from oracle import kv as okv

CASES = [(0.5, 1.0), (1e-3, 1.0), (1e-5, 1.0), (1.0, 1.0), (1.5, 0.1 * math.log(1.5) + 1),
         (16.0, 0.1 * math.log(16.0) + 1)]


@pytest.mark.parametrize("factor,magnitude", CASES)
def test_oracle(factor, magnitude):
    t = okv.table(2, 64, 10000.0, None, okv.YARN, factor, low=1.0, high=32.0, original=1024)
    assert np.allclose(np.hypot(t[..., 0], t[..., 1]), magnitude, rtol=1e-12)
    assert (t[0, :, 0] > 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("factor,magnitude", CASES)
def test_table(factor, magnitude):
    """A value is one rounding, 2^-24 of the magnitude; its angle is off by a few roundings of
    f64, 2^-48 of it."""
    rows, rot = 300, 64
    out = torch.empty(rows, rot // 2, 2, device="cuda")
    sc = wq.RopeScaling(wq.WQ_ROPE_YARN, 1024, factor, 1.0, 32.0, 0.0)
    wq.check(wq.wq_rope_table(rows, rot, 10000.0, sc, out), "wq_rope_table")
    got = out.cpu().double().numpy()
    f = okv.frequencies(rot, 10000.0, okv.YARN, factor, 1.0, 32.0, 1024)
    a = np.arange(rows)[:, None] * f
    want = magnitude * np.stack([np.cos(a), np.sin(a)], -1)
    assert (np.abs(got - want) <= 2.0 ** -24 * magnitude + 2.0 ** -48 * np.abs(a[..., None])).all()
