"""moe_kv_release, moe_kv_fork, moe_kv_reserve, moe_kv_compact and moe_kv_copy against their definitions, entry by entry: whole
numbers, so every table has to be equal."""
import random

import numpy as np
import pytest

import int4_routed_expert_02_amd as moe
from kv_pool_model import PoolModel

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.load()


def ints(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


class Pool:
    """The same state on the device; every call on outputs filled with garbage."""

    def __init__(self, m: PoolModel):
        self.m, self.n, self.width = m, len(m.pages), len(m.pages[0])
        self.push()

    def push(self):
        m = self.m
        self.pages, self.lens, self.slots, self.refs = ints(m.pages), ints(m.lens), ints(m.slots), ints(m.refs)

    def shape(self, rows=0, max_rows=0, max_len=1 << 30, window=0):
        return moe.kv_shape(self.n, rows, max_rows, max_len, 2, 2, 64, self.m.bits, self.m.P, self.m.n_pages, self.width,
                            self.n, window)

    def junk(self, n):
        import torch
        return torch.full((n,), 123456, dtype=torch.int32, device="cuda")

    def ws(self, sh):
        import torch
        return torch.full((moe.moe_kv_pool_workspace_bytes(sh),), 255, dtype=torch.uint8, device="cuda")

    def same(self, *pairs):
        m = self.m
        for got, want in ((self.pages, m.pages), (self.refs, m.refs), *pairs):
            got, want = got.cpu().numpy().reshape(-1), np.asarray(want, np.int64).reshape(-1)
            assert np.array_equal(got, want), (np.nonzero(got != want)[0][:5], got[got != want][:5], want[got != want][:5])

    def release(self, keep, window=0, sinks=0):
        moe.moe_kv_release(self.shape(window=window), sinks, ints(keep), self.pages, self.refs)
        self.m.release(keep, window, sinks)
        self.same()

    def fork(self, parent, slots=True):
        import torch
        out = [self.junk(self.n) for _ in range(4)]
        pages = torch.full_like(self.pages, 123456)
        bt = moe.kv_batch(ints([0] * (self.n + 1)), self.lens, self.pages, self.slots if slots else None)
        moe.moe_kv_fork(self.shape(), bt, ints(parent), out[0], pages, out[1], self.refs, out[2], out[3])
        src, dst = self.m.fork(parent)
        self.pages, self.lens = pages, out[0]
        if self.m.bits == 8:
            self.slots = out[1]
            self.same((self.lens, self.m.lens), (out[1], self.m.slots), (out[2], src), (out[3], dst))
        else:
            self.m.slots = list(range(self.n))
            self.same((self.lens, self.m.lens))
            assert (out[1] == 123456).all() and (out[2] == 123456).all()

    def reserve(self, new, max_len=1 << 30):
        sh = self.shape(sum(new), max(new), max_len)
        src, dst, missing = (self.junk(self.n) for _ in range(3))
        self.lens = self.lens + ints(new)
        bt = moe.kv_batch(ints(np.concatenate([[0], np.cumsum(new)])), self.lens, self.pages)
        moe.moe_kv_reserve(sh, bt, self.pages, self.refs, src, dst, missing, self.ws(sh))
        want = self.m.reserve(new, max_len)
        self.same((missing, want[2]), *(((src, want[0]), (dst, want[1])) if self.m.bits == 16 else ()))
        if self.m.bits == 8:
            assert (src == 123456).all()
        return want

    def compact(self, moves):
        src, dst, live = self.junk(moves), self.junk(moves), self.junk(1)
        sh = self.shape()
        moe.moe_kv_compact(sh, self.pages, self.refs, src, dst, live, self.ws(sh))
        want = self.m.compact(moves)
        self.same((src, want[0]), (dst, want[1]), (live, [want[2]]))


def walk(pool, rng, steps, most_new, max_len):
    """Calls in random order, as a server makes them."""
    m, n = pool.m, pool.n
    cap = min(max_len, pool.width * m.P)
    for _ in range(steps):
        kind = rng.choice(("reserve", "reserve", "reserve", "fork", "fork", "release", "drop", "compact"))
        if kind == "reserve":
            new = [0 if rng.random() < 0.2 else min(rng.randint(0, most_new), cap - a) for a in m.lens]
            pool.reserve(new)
        elif kind == "fork":
            pool.fork([rng.choice([s, rng.randrange(n), rng.randrange(max(1, n // 4)), -1 if rng.random() < 0.2 else s]) for s in range(n)])
        elif kind == "release":
            if rng.random() < 0.5:
                ended = [0 if rng.random() < 0.2 else a for a in m.lens]
                pool.release(ended)
                m.lens = ended
                pool.lens = ints(ended)
            else:
                pool.release(m.lens, rng.randint(1, 3 * m.P), rng.choice([0, 3, m.P, 2 * m.P + 1]))
        elif kind == "drop":                                      # tokens dropped: blocks behind the length stay in the table
            m.lens = [rng.randint(max(0, a - m.P), a) for a in m.lens]
            pool.lens = ints(m.lens)
        else:
            pool.compact(rng.choice([m.n_pages // 2, rng.randint(0, m.n_pages // 2)]))


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("seed", range(12))
def test_walk(seed, bits):
    """Few sequences and pages (every call in one launch), pools that run out among them."""
    rng = random.Random(seed * 2 + bits)
    n, page = rng.choice([1, 2, 7, 33, 100]), rng.choice([16, 32, 64, 128])
    width = rng.randint(1, 40)
    n_pages = max(1, int(n * width * rng.choice([0.2, 0.6, 1.5])))
    walk(Pool(PoolModel(n, width, page, n_pages, bits)), rng, 40, rng.choice([1, 5, 2 * page, 5 * page]), width * page)


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("n,width,n_pages", [(600, 5, 3000), (20, 300, 70001), (2, 9000, 20000), (1100, 20, 9000), (3, 70, 140001)])
def test_walk_large(n, width, n_pages, bits):
    """More sequences, blocks, entries or pages than the calls of one launch take."""
    rng = random.Random(n + bits)
    pool = Pool(PoolModel(n, width, 16, n_pages, bits))
    if n_pages > 60000:                                           # the lowest pages are taken: free ones are far up
        taken = rng.sample(range(n_pages - 200), n_pages - 400)
        for p in taken:
            pool.m.refs[p] = 1
        pool.push()
    walk(pool, rng, 14, rng.choice([16, 16 * width]), width * 16)


def test_many_sequences_in_a_reserve():
    """More sequences than a fork takes, one token each."""
    n = 20000
    pool = Pool(PoolModel(n, 3, 16, 50000, 16))
    pool.reserve([1] * n)
    pool.reserve([17] * n)
    pool.reserve([1 if s % 3 else 0 for s in range(n)])


def test_a_long_prompt():
    pool = Pool(PoolModel(3, 9000, 16, 30000, 8))
    pool.reserve([100000, 1, 70001])
    pool.fork([0, 0, 2])
    pool.reserve([1, 1, 43])
    pool.release([100000, 0, 50000])
    pool.compact(15000)


@pytest.mark.parametrize("bits", [8, 16])
def test_max_len(bits):
    """Only blocks below max_len and inside the table."""
    pool = Pool(PoolModel(4, 6, 16, 40, bits))
    pool.reserve([50, 30, 0, 96], max_len=40)
    pool.reserve([46, 80, 200, 300], max_len=1 << 30)


@pytest.mark.parametrize("bits", [8, 16])
def test_largest_fork(bits):
    rng = random.Random(bits)
    n = moe.MOE_KV_FORK_MAX
    pool = Pool(PoolModel(n, 3, 16, 2 * n, bits))
    pool.reserve([rng.randint(0, 20) for _ in range(n)])
    pool.fork([rng.randrange(-5, n + 5) for _ in range(n)])
    pool.fork([17] * n)
    pool.reserve([1] * n)


def test_without_slots():
    """8 bits without a table of slots: sequence s has slot s."""
    pool = Pool(PoolModel(6, 4, 16, 40, 8))
    pool.reserve([20, 0, 5, 33, 1, 16])
    pool.fork([3, 3, 0, -1, 5, 3], slots=False)


@pytest.mark.parametrize("n_pages", [50, 70001])
def test_ids_outside_the_cache(n_pages):
    """Tables that hold ids outside the cache name no page with them; counts below 0 are free pages."""
    m = PoolModel(5, 8, 16, n_pages, 16)
    rng = random.Random(n_pages)
    for row in m.pages:
        for b in range(8):
            row[b] = rng.choice([-1, -2 ** 31, 2 ** 31 - 1, n_pages, n_pages + 5, rng.randrange(n_pages)])
            if m.valid(row[b]):
                m.refs[row[b]] += 1
    m.refs[1] = -3 if m.refs[1] == 0 else m.refs[1]
    m.lens = [0, 5, 128, 77, 128]
    pool = Pool(m)
    pool.reserve([1, 20, 0, 51, 0])
    pool.fork([2, 2 ** 31 - 1, -2 ** 31, 3, 1])
    pool.compact(n_pages // 2)
    pool.release([3, 0, 0, 100, 2 ** 30])


@pytest.mark.parametrize("n,n_pages", [(30, 500), (2000, 500), (2000, 90000)])
def test_rows_that_do_not_ascend(n, n_pages):
    """A table of rows that makes no sense: the call ends, and every entry and list names pages of the cache or none."""
    rs = np.random.RandomState(n)
    pool = Pool(PoolModel(n, 20, 16, n_pages, 16))
    sh = pool.shape(3000, 3000)
    src, dst, missing = (pool.junk(n) for _ in range(3))
    for starts in (rs.randint(-5, 4000, n + 1), np.where(np.arange(n + 1) % 2, 3000, 0), np.arange(n + 1)[::-1]):
        bt = moe.kv_batch(ints(starts), ints(rs.randint(-5, 400, n)), pool.pages)
        moe.moe_kv_reserve(sh, bt, pool.pages, pool.refs, src, dst, missing, pool.ws(sh))
        for t in (pool.pages, src, dst):
            assert int(t.min()) >= -1 and int(t.max()) < n_pages


def test_one_page_twice():
    """A row, or two rows, that name a page twice: it counts as often, and is parted like any other."""
    for bits in (8, 16):
        m = PoolModel(3, 4, 16, 20, bits)
        m.pages[0][:2] = [7, 7]
        m.pages[1][:2] = [7, 9]
        m.pages[2][:3] = [9, 9, 9]
        m.refs[7], m.refs[9] = 3, 4
        m.lens = [16, 16, 0]
        pool = Pool(m)
        pool.reserve([5, 5, 48])
        pool.fork([0, 0, 2])
        pool.release([0, 20, 16])


def test_nothing_to_do():
    import torch
    pool = Pool(PoolModel(4, 5, 16, 30, 16))
    pool.reserve([3, 0, 17, 0])
    pool.reserve([0, 0, 0, 0])                                    # rows 0: the lists are written all the same
    pool.compact(0)
    m = PoolModel(2, 3, 16, 0, 16)                                # a cache without pages
    empty = Pool(m)
    empty.reserve([5, 20])
    empty.fork([1, 1])
    empty.release([0, 0])
    empty.compact(0)
    sh = moe.kv_shape(0, 0, 0, 10, 2, 2, 64, 16, 16, 30, 5, 0)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    moe.moe_kv_release(sh, 0, none, none, pool.refs)
    src = ints([5] * 15)
    moe.moe_kv_compact(sh, none, pool.refs, src, ints([5] * 15), None, pool.ws(sh))
    assert (src == -1).all()                                      # no hole below the pages in use


# ---------------------------------------------------------------- copies


def filled(n_pages, heads, dim, page, bits, slots, seed=0):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = moe.KvPages(n_pages, heads, dim, page, bits, slots)
    for t in (c.k, c.v, c.k_scale, c.v_scale, c.k_tail, c.v_tail):
        if t is not None:
            t.copy_(torch.randint(-120, 120, t.shape, generator=g, device="cuda"))
    return c


def tensors(c):
    return {n: getattr(c, n) for n in ("k", "v", "k_scale", "v_scale", "k_tail", "v_tail") if getattr(c, n) is not None}


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("heads,dim,page", [(1, 64, 16), (3, 64, 16), (4, 64, 64), (8, 128, 128), (300, 64, 16)])
@pytest.mark.parametrize("n", [1, 5, 700])
def test_copy(n, heads, dim, page, bits):
    import torch
    rs = np.random.RandomState(n + heads)
    n_pages, n_slots = 2 * n + 3, (2 * min(n, 20) + 1 if bits == 8 else 0)
    c = filled(n_pages, heads, dim, page, bits, n_slots)
    want = {k: t.clone() for k, t in tensors(c).items()}
    lists = []
    for total, count, names in ((n_pages, n, ("k", "v", "k_scale", "v_scale")), (n_slots, min(n, 20), ("k_tail", "v_tail"))):
        if total == 0:
            lists += [None, None]
            continue
        ids = rs.permutation(total)
        src, dst = ids[:count].astype(np.int64), ids[count:2 * count].astype(np.int64)
        src[rs.rand(count) < 0.2] = -1
        if count > 4:
            src[0], dst[1], src[2], dst[3] = total, -1, -2 ** 31, 2 ** 31 - 1
            src[4] = dst[4]
        for a, b in zip(src, dst):
            if 0 <= a < total and 0 <= b < total:
                for k in names:
                    if k in want:
                        want[k][b] = want[k][a]
        lists += [ints(src), ints(dst)]
    sh = c.shape(0, 0, 0, 0, heads, 0)
    moe.moe_kv_copy(sh, c.handle, *lists)
    for k, t in tensors(c).items():
        assert torch.equal(t, want[k]), k
    moe.moe_kv_copy(sh, c.handle)                                 # no list
    for k, t in tensors(c).items():
        assert torch.equal(t, want[k]), k


def test_copy_far():
    """Pages whose offsets pass 32 bits."""
    import torch
    n_pages, H, D, P = 40000, 8, 128, 128                         # 5.2e9 values of K
    c = moe.KvPages(n_pages, H, D, P, 8, 1)
    c.k_scale.zero_()
    src, dst = [n_pages - 1, 5, 33333], [3, n_pages - 2, 17000]
    for i, p in enumerate(src):
        c.k[p], c.v[p], c.k_scale[p] = i + 1, -i - 1, i + 0.5
    moe.moe_kv_copy(c.shape(0, 0, 0, 0, H, 0), c.handle, ints(src), ints(dst))
    for i, p in enumerate(dst):
        assert (c.k[p] == i + 1).all() and (c.v[p] == -i - 1).all() and (c.k_scale[p] == i + 0.5).all()
