"""Workspaces of the paged-cache calls: never empty for valid arguments, and refused when
missing, misaligned or a byte short (CPU only)."""
import pytest

import gemv_transformer_gb300 as wq
from test_kv_abi import A, BAD, attn, cache, evict, lib  # noqa: F401


@pytest.mark.parametrize("n,hq,wide", [(1, 2, 1), (2, 4, 4), (64, 16, 100), (500, 40, 3)])
@pytest.mark.parametrize("kind", [wq.WQ_BF16, wq.WQ_F16, wq.WQ_F32])
@pytest.mark.parametrize("with_acc", [0, 1])
def test_attention(n, hq, wide, kind, with_acc):
    c = cache(dtype=kind)
    need = wq.wq_attn_paged_workspace_bytes(c, n, hq, wide, with_acc)
    # The weight sums keep every score.
    assert need > with_acc * 4 * n * hq * wide * 16
    kw = dict(c=c, n=n, hq=hq, qs=hq * 64, os=hq * 64, wide=wide, aout=A if with_acc else None, st=64)
    assert attn(room=None, size=need, **kw) == BAD
    assert attn(room=A + 16, size=need, **kw) == BAD
    assert attn(size=need - 1, **kw) == BAD
    assert attn(size=0, **kw) == BAD


@pytest.mark.parametrize("n,wide,keep", [(1, 1, 1), (2, 4, 8), (64, 100, 1000), (3, 4, 10 ** 6)])
def test_eviction(n, wide, keep):
    need = wq.wq_kv_evict_workspace_bytes(cache(), n, wide, keep)
    assert need >= n * 2 * min(keep, wide * 16) * 8
    kw = dict(n=n, wide=wide, keep=keep)
    assert evict(room=None, size=need, **kw) == BAD
    assert evict(room=A + 16, size=need, **kw) == BAD
    assert evict(size=need - 1, **kw) == BAD
