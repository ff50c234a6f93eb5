"""Shared by the tests of the calls for several new tokens per sequence."""
from __future__ import annotations

import numpy as np
import torch

import gemv_transformer_gb300 as wq
from helpers import dev

KINDS = {"bf16": wq.WQ_BF16, "f16": wq.WQ_F16, "f32": wq.WQ_F32}
TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# Half a step of a type, relative to the value.
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}


def as_type(x, kind):
    """A device tensor of the type, and the values that it holds in f64."""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(TORCH[kind])
    return t.cuda(), t.double().numpy()


def angles(rows, pairs, base=10000.0):
    """A table [rows][pairs][2] in f32."""
    f = base ** (-np.arange(pairs) / pairs)
    a = np.arange(rows)[:, None] * f
    return np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)


def random_tree(g, count):
    """Parents, and for each node the set of nodes at and above it."""
    parent = [-1] + [int(g.integers(max(0, j - 4), j)) for j in range(1, count)]
    above = []
    for j in range(count):
        above.append({j} | (above[parent[j]] if j else set()))
    return parent[:count], above


def tree_words(rows, words):
    """int32 [tokens][words] of sets of nodes."""
    out = np.zeros((len(rows), words), np.uint32)
    for t, nodes in enumerate(rows):
        for b in nodes:
            out[t, b // 32] |= np.uint32(1 << (b % 32))
    return dev(out.view(np.int32))
