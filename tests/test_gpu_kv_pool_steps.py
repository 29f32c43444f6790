"""Pools of more pages than the workgroups over the counts take in one step each (8192 blocks of 4096 pages): only the tables and
the counts are there, against the sequential model.  What the model would go through page by page in Python it gets as the few
pages that are free or in use."""
import numpy as np
import pytest

import int4_routed_expert_02_amd as moe

pytestmark = pytest.mark.gpu

N_PAGES = 8192 * 4096 * 2 + 777                                 # three steps a workgroup


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.load()


def ints(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def test_reserve_takes_the_lowest_free_pages():
    """All pages in use but for a few near the borders of blocks and steps; a pool that runs out at last."""
    import torch
    free = sorted({0, 5, 4095, 4096, 8191, 12287, 12288, 3 * 4096 * 17 + 1, 8192 * 4096 - 1, 8192 * 4096, N_PAGES // 2, N_PAGES - 778,
                   N_PAGES - 777, N_PAGES - 2, N_PAGES - 1})
    refs = torch.ones(N_PAGES, dtype=torch.int32, device="cuda")
    refs[torch.tensor(free, device="cuda")] = 0
    n = 4
    pages, lens = torch.full((n, 8), -1, dtype=torch.int32, device="cuda"), ints([0] * n)
    missing, lists = ints([9] * n), [ints([9] * n) for _ in range(2)]
    left, held = list(free), [[] for _ in range(n)]
    for new in ([16, 33, 0, 1], [1, 0, 16, 16], [78, 0, 64, 0]):
        sh = moe.kv_shape(n, sum(new), max(new), 128, 1, 1, 64, 16, 16, N_PAGES, 8)
        ws = torch.full((moe.moe_kv_pool_workspace_bytes(sh),), 255, dtype=torch.uint8, device="cuda")
        lens += ints(new)
        moe.moe_kv_reserve(sh, moe.kv_batch(ints(np.concatenate([[0], np.cumsum(new)])), lens, pages), pages, refs, *lists, missing, ws)
        lacks = [0] * n
        for s in range(n):
            for _ in range(-(-int(lens[s]) // 16) - len(held[s])):
                held[s].append(left.pop(0) if left else -1)
                lacks[s] += held[s][-1] < 0
        assert missing.tolist() == lacks
        for s in range(n):
            assert pages[s].tolist() == held[s] + [-1] * (8 - len(held[s]))
        assert (lists[0] == -1).all() and (lists[1] == -1).all()
    taken = [p for row in held for p in row if p >= 0]
    assert not left and sorted(taken) == free
    assert bool((refs == 1).all())


@pytest.mark.parametrize("moves", [3, 20])
def test_compact_moves_from_far(moves):
    """Few pages in use, the highest ones among them, and a hole or two below."""
    import torch
    used = [1, 2, 9, 4097, 8192 * 4096 - 1, 8192 * 4096 + 3, N_PAGES - 778, N_PAGES - 777, N_PAGES - 1]
    order = np.random.RandomState(0).permutation(len(used))
    refs = torch.zeros(N_PAGES, dtype=torch.int32, device="cuda")
    table = np.full((3, 7), -1)
    table.reshape(-1)[[0, 2, 3, 8, 9, 10, 15, 19, 20]] = np.asarray(used)[order]
    table[2, 2] = used[-1]                                        # shared
    pages = ints(table)
    for p in table.reshape(-1):
        if p >= 0:
            refs[int(p)] += 1
    sh = moe.kv_shape(3, 0, 0, 112, 1, 1, 64, 16, 16, N_PAGES, 7)
    src, dst, live = ints([9] * moves), ints([9] * moves), ints([9])
    ws = torch.full((moe.moe_kv_pool_workspace_bytes(sh),), 255, dtype=torch.uint8, device="cuda")
    moe.moe_kv_compact(sh, pages, refs, src, dst, live, ws)
    n = len(used)
    pairs = list(zip([p for p in reversed(used) if p >= n], [p for p in range(n) if p not in used]))[:moves]
    pad = [-1] * (moves - len(pairs))
    assert int(live) == n and src.tolist() == [a for a, _ in pairs] + pad and dst.tolist() == [b for _, b in pairs] + pad
    to = dict(pairs)
    want = np.vectorize(lambda p: to.get(int(p), int(p)))(table)
    assert pages.tolist() == want.tolist()
    counts = torch.bincount(pages[pages >= 0].long(), minlength=N_PAGES)
    assert torch.equal(counts.int(), refs)
