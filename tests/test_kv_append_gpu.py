"""GPU parity of wq_kv_append: queries and keys rotated (f64 oracle), keys and values in
their pages, everything else untouched.

Tolerances: q as wq_rope, 2^-22 of its terms; a cached key is the rounding to the cache's type
of a value that near the oracle's: it lies between the roundings of that range's two ends
(rounding is monotone).  Values are copied: the same bits as torch's rounding."""
import numpy as np
import pytest
import torch

import gemv_transformer_gb300 as wq
from helpers import Guarded, dev, status_ok
from kv_helpers import Cache, bits
from oracle import kv as okv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from gemv_transformer_gb300 import build
    build.build()
    wq.load()
    yield
    status_ok()


def run_append(seed, n_seq, lens, hq, hkv, d, rot, seq, slot, kind="bf16", page=16, major="head",
               flags=0, acc=True, rows=400, pos=None, in_place=False, shift=0, status=wq.WQ_OK,
               spoil=None):
    g = np.random.default_rng(seed)
    c = Cache(g, lens, hkv, d, kind, page, major)
    if spoil:
        spoil(c)
    m = len(slot)
    width = (hq + 2 * hkv) * d + shift
    qkv = torch.randn(m * width + shift, generator=torch.Generator().manual_seed(seed)).cuda()
    qkv = qkv[shift:].view(m, width)
    x = qkv[:, :(hq + 2 * hkv) * d].cpu().view(m, hq + 2 * hkv, d)
    pos = g.integers(0, rows, m).astype(np.int32) if pos is None else np.asarray(pos, np.int32)
    table = torch.empty(rows * max(rot, 2), device="cuda")
    wq.check(wq.wq_rope_table(rows, max(rot, 2), 10000.0, None, table))
    cap = c.max_pages * page
    sums = torch.full((n_seq, hkv, cap), 7.0, device="cuda") if acc else None
    at = torch.full((n_seq, hkv, cap), -9, dtype=torch.int32, device="cuda") if acc else None
    out = Guarded(m * hq * d, np.full(m * hq * d, 5.0, np.float32))
    before = [p.clone() for p in c.pools]
    q_out, q_stride = (qkv, width) if in_place else (out.view, hq * d)
    wq.check(wq.wq_kv_append(
        c.desc, m, hq, rot, flags, qkv if hq else None, width, qkv[:, hq * d:], width,
        qkv[:, (hq + hkv) * d:], width, dev(pos), table if rot else None, rows, n_seq,
        None if seq is None else dev(np.asarray(seq, np.int32)), dev(np.asarray(slot, np.int32)),
        c.pages_dev, c.max_pages, q_out if hq else None, q_stride, sums, at, cap), "wq_kv_append")
    torch.cuda.synchronize()
    assert wq.wq_get_device_status() == status
    if in_place:
        q = qkv[:, :hq * d].cpu().numpy().reshape(m, hq, d)
    else:
        q = out.result().reshape(m, hq, d)
    cs = table.cpu().numpy().astype(np.float64).reshape(rows, -1, 2)
    want, mag = okv.rotate(x[:, :hq + hkv].numpy(), cs[np.clip(pos, 0, rows - 1)], rot, flags)
    k_now, v_now = (p.cpu() for p in c.pools)
    k_was, v_was = (p.cpu() for p in before)
    written = torch.zeros(k_now.shape[:3], dtype=torch.bool)
    s_now = sums.cpu().numpy() if acc else None
    p_now = at.cpu().numpy() if acc else None
    for t in range(m):
        s, j = (t if seq is None else seq[t]), slot[t]
        ok = 0 <= s < n_seq and 0 <= j < cap and (rot == 0 or 0 <= pos[t] < rows)
        page_id = c.pages[s, j // page] if ok else -1
        ok = ok and 0 <= page_id < k_now.shape[0]
        if not ok:
            if not in_place:
                assert (q[t] == 5.0).all()
            continue
        assert (np.abs(q[t] - want[t, :hq]) <= 2.0 ** -22 * mag[t, :hq]).all()
        got = k_now[page_id, :, j % page].double().numpy()
        w, b = want[t, hq:], mag[t, hq:]
        lo, hi = (torch.from_numpy(w + e * 2.0 ** -22 * b).to(k_now.dtype).double().numpy()
                  for e in (-1, 1))
        assert (lo <= got).all() and (got <= hi).all()
        v_want = x[t, hq + hkv:].to(v_now.dtype)
        assert np.array_equal(bits(v_now[page_id, :, j % page]), bits(v_want))
        written[page_id, :, j % page] = True
        if acc:
            assert (s_now[s, :, j] == 0).all() and (p_now[s, :, j] == pos[t]).all()
            s_now[s, :, j], p_now[s, :, j] = 7.0, -9
    for now, was in ((k_now, k_was), (v_now, v_was)):
        assert np.array_equal(bits(now[~written]), bits(was[~written]))
    if acc:
        assert (s_now == 7.0).all() and (p_now == -9).all()
    return c


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("hq,hkv,d,rot,page,major", [
    (8, 2, 128, 128, 16, "head"), (1, 1, 64, 64, 1, "token"), (5, 5, 80, 40, 7, "gap"),
    (32, 8, 96, 96, 64, "token"), (0, 3, 72, 36, 16, "head"), (4, 1, 256, 128, 3, "token"),
    (2, 1, 8, 0, 5, "head")])
@pytest.mark.parametrize("flags", [0, wq.WQ_ROPE_INTERLEAVED])
def test_one_token_of_each_sequence(kind, hq, hkv, d, rot, page, major, flags):
    lens = [1, 16, 33, 50, 7]
    run_append(d + rot, 5, lens, hq, hkv, d, rot, None, [n - 1 for n in lens], kind, page, major,
               flags)


@pytest.mark.parametrize("in_place,shift", [(True, 0), (False, 1), (True, 3), (False, 4)])
def test_prompts_of_several_sequences(in_place, shift):
    lens = [40, 3, 111]
    seq = [0] * 40 + [1] * 3 + [2] * 100
    slot = list(range(40)) + list(range(3)) + list(range(11, 111))
    order = np.random.default_rng(1).permutation(len(seq))
    run_append(11, 3, lens, 4, 2, 128, 128, [seq[i] for i in order], [slot[i] for i in order],
               in_place=in_place, shift=shift, acc=not shift)


def test_padding_and_indices_out_of_range():
    """A negative slot is padding (no error); the other tokens that are left out are."""
    lens = [20, 20]
    run_append(12, 2, lens, 2, 1, 64, 64, [0, 1, 0], [3, -1, 19])
    run_append(13, 2, lens, 2, 1, 64, 64, [0, 2, 1, -1, 0], [0, 0, 32, 1, 19],
               status=wq.WQ_ERR_BAD_INDEX)
    run_append(14, 2, lens, 2, 1, 64, 64, [0, 1, 0], [0, 1, 2], pos=[400, -1, 399],
               status=wq.WQ_ERR_BAD_INDEX)

    def spoil(c):  # a page beyond the pool, and one that is not there
        c.pages[0, 0], c.pages[1, 1] = c.pools[0].shape[0], -1
        c.pages_dev = dev(c.pages)
    run_append(15, 2, lens, 2, 1, 64, 64, [0, 0, 1, 1], [0, 19, 5, 17], spoil=spoil,
               status=wq.WQ_ERR_BAD_INDEX)


def test_pages_beyond_4_gib():
    """Pages whose byte offsets pass 2^32."""
    pages, hkv, page, d = 5, 2, 16, 128
    stride = (1 << 30) + 64  # elements: 2 GiB and a little per page
    room = torch.empty(pages * stride, dtype=torch.bfloat16, device="cuda")
    view = room.as_strided((pages, hkv, page, d), (stride, page * d, d, 1))
    view.fill_(0)
    g = torch.Generator().manual_seed(3)
    x = torch.randn(80, 2 * hkv * d, generator=g)
    table = np.array([[4, 2, 0, 3, 1]], np.int32)
    xd = x.cuda()
    cache = wq.kv_cache(view, view)  # one pool for both: the call writes keys, then nothing else
    cache.v = view.data_ptr() + 2 * hkv * page * d  # values after a page's keys
    wq.check(wq.wq_kv_append(cache, 80, 0, 0, 0, None, 0, xd, 2 * hkv * d, xd[:, hkv * d:],
                             2 * hkv * d, None, None, 0, 1, dev(np.zeros(80, np.int32)),
                             dev(np.arange(80, dtype=np.int32)), dev(table), 5))
    torch.cuda.synchronize()
    both = room.as_strided((pages, 2, hkv, page, d),
                           (stride, hkv * page * d, page * d, d, 1))
    for t in (0, 17, 40, 50, 79):
        want = x[t].view(2, hkv, d).to(torch.bfloat16)
        got = both[table[0, t // 16], :, :, t % 16].cpu()
        assert torch.equal(got, want)
