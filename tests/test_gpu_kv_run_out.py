"""A pool that runs out in the middle of a shared page: what the sequence without a page loses, and that a program which puts the
tables back, ends another sequence and calls again loses nothing.  All comparisons are of bits."""
import pytest

import int4_routed_expert_02_amd as moe
from test_gpu_kv_serving import Server, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.load()


def full(bits, layers=2):
    """Sequences 0 and 1 share three pages, the last with eight rows; sequence 2 has the pool's other two."""
    s = Server(3, 16, bits, 5, 4, layers=layers, seed=4)
    s.append([40, 0, 30])
    s.fork([0, 0, 2])
    return s


def reserve(s, new):
    """As before an append of `new` rows: the lists and the counts of blocks without a page."""
    import torch
    starts = ints([0, new[0], new[0] + new[1], sum(new)])
    sh = s.shape(s.caches[0], sum(new), max(new))
    ws = torch.empty(moe.moe_kv_pool_workspace_bytes(sh), dtype=torch.uint8, device="cuda")
    lens = s.lens + ints(new)
    moe.moe_kv_reserve(sh, moe.kv_batch(starts, lens, s.pages, s.slots), s.pages, s.refs, *s.lists[2:], s.missing, ws)
    return s.missing.tolist()


@pytest.mark.parametrize("bits", [8, 16])
def test_what_is_lost(bits):
    """The first of the sharers keeps the page, the other has none from then on, also when pages are free again."""
    s = full(bits)
    page = int(s.pages[0, 2])
    assert reserve(s, [1, 1, 0]) == [0, 1, 0]
    assert int(s.pages[0, 2]) == page and int(s.pages[1, 2]) == -1 and int(s.refs[page]) == 1
    s.release(ints([41, 41, 0]))
    assert reserve(s, [1, 1, 0]) == [0, 1, 0]
    assert int(s.pages[1, 2]) == -1


@pytest.mark.parametrize("bits", [8, 16])
def test_tables_put_back(bits):
    s = full(bits)
    kept = s.pages.clone(), s.refs.clone()

    def put_back():
        s.pages.copy_(kept[0])
        s.refs.copy_(kept[1])

    assert reserve(s, [9, 9, 0]) == [1, 2, 0]                    # a new block each, and the page that one of the two gives up
    put_back()
    s.check(None, None)
    s.release(ints([40, 40, 0]))                                 # sequence 2 ends
    s.lens[2], s.history[2] = 0, []
    kept = s.pages.clone(), s.refs.clone()
    assert reserve(s, [9, 9, 0]) == [0, 1, 0]                    # still one too few
    put_back()
    got = s.append([8, 8, 0])                                    # to the end of the page: one more page is enough
    assert s.missing.tolist() == [0, 0, 0]
    s.check([8, 8, 0], got)
    got = s.append([1, 0, 0])
    assert s.missing.tolist() == [0, 0, 0]
    s.check([1, 0, 0], got)
