"""What wq_kv_accept leaves alone where indexes are out of range: every pool bit for bit."""
import numpy as np
import pytest

import gemv_transformer_gb300 as wq
from helpers import status_ok
from kv_helpers import bits
from oracle import tokens as ot
from test_kv_accept_gpu import Draft

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from gemv_transformer_gb300 import build
    build.build()
    wq.load()
    yield
    status_ok()


def rows(pool):
    return bits(pool).reshape(pool.shape[:3] + (-1,)).copy()


def run_and_compare(d, pages, nodes, skip=lambda s, slot: False):
    """Runs the call; the pools are as before but for the moves of `nodes`."""
    before = [[rows(p) for p in c.pools] for c in d.caches]
    moved = 0
    d.run()
    assert wq.wq_get_device_status() == wq.WQ_ERR_BAD_INDEX
    for c, pools in zip(d.caches, before):
        for pool, old in zip(c.pools, pools):
            want = old.copy()
            for s, chain in enumerate(nodes):
                b = d.lens[s] - d.counts[s]
                for i, node in enumerate(chain):
                    src, dst = b + node, b + i
                    if skip(s, src) or skip(s, dst):
                        continue
                    moved += src != dst
                    want[pages[s, dst // d.page], :, dst % d.page] = \
                        old[pages[s, src // d.page], :, src % d.page]
            assert (rows(pool) == want).all()
    return moved


@pytest.mark.parametrize("kind,page", [("bf16", 16), ("f32", 7)])
def test_refused_sequences_keep_their_slots(kind, page):
    """Starts that fall, a length beyond the pages, one below the nodes: only the first moves."""
    d = Draft(6, [20, 30, 10, 5], [40, 12, 3, 2], 2, kind=kind, page=page, agree=1.0)
    first = ot.accept(d.starts[:2], d.parent[:20], d.tokens[:20], d.choice[:20], d.lens[:1])
    d.starts = np.array([0, 20, 15, 60, 65], np.int32)
    d.lens[2], d.lens[3] = 10 ** 6, 4
    assert run_and_compare(d, d.pages, [first[4][0], [], [], []]) > 0
    assert d.path.tolist()[:20] == first[0].tolist() and (d.path[20:] == 77).all()
    assert d.accepted.tolist()[:4] == [first[1][0], 0, 0, 0]
    assert d.lens_out.tolist()[:4] == [first[3][0], 42, 10 ** 6, 4]


@pytest.mark.parametrize("bad", [-1, 10 ** 6])
@pytest.mark.parametrize("which", [1, 4])
def test_nodes_of_a_page_out_of_range_stay(bad, which):
    """The page of the path's `which`-th node: what comes from it or would go to it stays, the rest
    moves."""
    d = Draft(9, [40], [40], 2, agree=1.0, page=4)
    nodes = ot.accept(d.starts, d.parent, d.tokens, d.choice, d.lens)[4]
    lost, pages = (40 + nodes[0][which]) // 4, d.pages
    d.pages = pages.copy()
    d.pages[0, lost] = bad
    assert run_and_compare(d, pages, nodes, lambda s, slot: slot // 4 == lost) > 0
    assert d.accepted.tolist()[0] == len(nodes[0])
    assert d.path.tolist()[:len(nodes[0])] == nodes[0]
