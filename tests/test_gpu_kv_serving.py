"""The calls on a cache's pages together with append and attention, as a server makes them: beams that fork, share pages, write,
drop tokens, leave windows behind and end, against sequences that each have all of their pages alone.

The stored values and the attention over them do not depend on which page holds what, so all comparisons are of bits."""
import random

import numpy as np
import pytest

import int4_routed_expert_02_amd as moe
from kv_testutil import poison

pytestmark = pytest.mark.gpu

HQ, H, D = 8, 2, 64
QUERIES = {}  # by the number of rows


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.load()


def ints(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


class Server:
    """n sequences over one pool, `layers` caches with the same tables; what each sequence was given, on the host."""

    def __init__(self, n, page, bits, n_pages, width, window=0, sinks=0, layers=1, seed=0):
        import torch
        self.n, self.P, self.bits, self.width, self.window, self.sinks = n, page, bits, width, window, sinks
        self.caches = [moe.KvPages(n_pages, H, D, page, bits, n if bits == 8 else 0) for _ in range(layers)]
        for c in self.caches:
            poison(c)
        self.pages = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
        self.pages2, self.refs = torch.full_like(self.pages, 99), torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        self.lens, self.lens2 = ints([0] * n), ints([99] * n)
        self.slots, self.slots2 = ints(np.random.RandomState(seed).permutation(n)), ints([99] * n)
        self.lists = [ints([99] * n) for _ in range(4)]
        self.missing = ints([99] * n)
        self.moves = [ints([99] * (n_pages // 2)) for _ in range(2)]
        self.parent, self.starts = ints(range(n)), ints([0] * (n + 1))
        self.history = [[] for _ in range(n)]                    # per token: one row of k and v of each layer
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def shape(self, cache, rows=0, max_rows=0):
        return cache.shape(self.n, rows, max_rows, self.width * self.P, HQ, self.width, window=self.window)

    def fork(self, parent):
        self.parent.copy_(ints(parent))
        self.enqueue_fork()
        self.history = [list(self.history[p]) if 0 <= p < self.n else [] for p in parent]

    def enqueue_fork(self):
        sh = self.shape(self.caches[0])
        bt = moe.kv_batch(self.starts, self.lens, self.pages, self.slots)
        moe.moe_kv_fork(sh, bt, self.parent, self.lens2, self.pages2, self.slots2, self.refs, *self.lists[:2])
        self.pages.copy_(self.pages2)
        self.lens.copy_(self.lens2)
        if self.bits == 8:
            self.slots.copy_(self.slots2)
            for c in self.caches:
                moe.moe_kv_copy(sh, c.handle, slot_src=self.lists[0], slot_dst=self.lists[1])

    def rows(self, count):
        import torch
        return torch.randn(count, len(self.caches), 2, H, D, generator=self.g, device="cuda").to(torch.bfloat16)

    def append(self, new):
        """`new[s]` random rows for each sequence; the attention's outputs of the first layer."""
        starts = np.concatenate([[0], np.cumsum(new)])
        kv = self.rows(int(starts[-1]))
        for s in range(self.n):
            self.history[s] += [kv[r] for r in range(starts[s], starts[s + 1])]
        self.lens += ints(new)
        return self.enqueue_append(kv, ints(starts), int(starts[-1]), max(new))

    def enqueue_append(self, kv, starts, rows, most):
        import torch
        bt = moe.kv_batch(starts, self.lens, self.pages, self.slots)
        sh = self.shape(self.caches[0], rows, most)
        ws = torch.empty(moe.moe_kv_pool_workspace_bytes(sh), dtype=torch.uint8, device="cuda")
        moe.moe_kv_reserve(sh, bt, self.pages, self.refs, *self.lists[2:], self.missing, ws)
        for i, c in enumerate(self.caches):
            if self.bits == 16:
                moe.moe_kv_copy(sh, c.handle, page_src=self.lists[2], page_dst=self.lists[3])
            if rows:
                moe.moe_kv_append(sh, bt, c.handle, kv[:, i, 0].contiguous(), kv[:, i, 1].contiguous())
        return self.attend(sh, bt, self.caches[0], rows) if rows else None

    def attend(self, sh, bt, cache, rows):
        import torch
        if rows not in QUERIES:
            QUERIES[rows] = torch.randn(rows, HQ, D, generator=torch.Generator(device="cuda").manual_seed(rows), device="cuda").to(torch.bfloat16)
        q = QUERIES[rows]
        out, lse = torch.empty_like(q), torch.empty(rows, HQ, device="cuda")
        ws = torch.empty(moe.moe_kv_attention_sinks_workspace_bytes(sh, self.sinks), dtype=torch.uint8, device="cuda")
        moe.moe_kv_attention_sinks(sh, self.sinks, bt, cache.handle, q, out, lse, ws)
        return out, lse

    def release(self, keep=None):
        moe.moe_kv_release(self.shape(self.caches[0]), self.sinks, self.lens if keep is None else keep, self.pages, self.refs)

    def compact(self):
        import torch
        sh = self.shape(self.caches[0])
        ws = torch.empty(moe.moe_kv_pool_workspace_bytes(sh), dtype=torch.uint8, device="cuda")
        moe.moe_kv_compact(sh, self.pages, self.refs, *self.moves, None, ws)
        for c in self.caches:
            moe.moe_kv_copy(sh, c.handle, page_src=self.moves[0], page_dst=self.moves[1])

    def check(self, new, got):
        """The same histories in caches of their own, each appended at once; the last `new` rows' attention over them."""
        import torch
        lens = [len(h) for h in self.history]
        assert self.lens.tolist() == lens
        named = self.pages[(self.pages >= 0)]
        assert torch.equal(torch.bincount(named.long(), minlength=self.refs.numel()), self.refs.long())
        if not sum(lens):
            return
        for i in range(len(self.caches)):
            own = moe.KvPages(self.n * self.width, H, D, self.P, self.bits, self.n if self.bits == 8 else 0)
            poison(own)
            ids = torch.arange(self.n * self.width, dtype=torch.int32, device="cuda").view(self.n, self.width)
            bt = moe.kv_batch(ints(np.concatenate([[0], np.cumsum(lens)])), self.lens, ids)
            kv = torch.stack([r for h in self.history for r in h])[:, i]
            sh = self.shape(own, sum(lens), max(lens))
            moe.moe_kv_append(sh, bt, own.handle, kv[:, 0].contiguous(), kv[:, 1].contiguous())
            if new is not None and i == 0 and sum(new):
                part = moe.kv_batch(ints(np.concatenate([[0], np.cumsum(new)])), self.lens, ids)
                want = self.attend(self.shape(own, sum(new), max(new)), part, own, sum(new))
                for a, b in zip(got, want):
                    assert torch.equal(a.view(torch.int16 if a.dtype == torch.bfloat16 else torch.int32),
                                       b.view(torch.int16 if b.dtype == torch.bfloat16 else torch.int32))
            # what the shared cache holds, where a later row can see it
            mine = self.caches[i]
            there = moe.kv_batch(bt.tensors[0], self.lens, self.pages, self.slots)
            read = []
            for cache, batch in ((mine, there), (own, bt)):
                k, v = (torch.empty(sum(lens), H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
                moe.moe_kv_read(self.shape(cache, sum(lens), max(lens)), batch, cache.handle, k, v)
                read.append((k, v))
            seen = np.concatenate([(np.arange(n) >= n - self.window + 1 if self.window else np.ones(n, bool)) | (np.arange(n) < self.sinks)
                                   for n in lens])
            seen = torch.from_numpy(seen).cuda()
            for a, b in zip(*read):
                assert torch.equal(a[seen].view(torch.int16), b[seen].view(torch.int16))


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("window,sinks", [(0, 0), (37, 5), (100, 64)])
@pytest.mark.parametrize("seed", range(3))
def test_beams(seed, window, sinks, bits):
    rng = random.Random(seed)
    n, page = rng.choice([4, 6, 9]), rng.choice([16, 32, 64])
    width = -(-400 // page)
    s = Server(n, page, bits, 2 * n * width, width, window, sinks, layers=rng.choice([1, 2]), seed=seed)
    prompts = [rng.choice([0, rng.randint(1, 150)]) for _ in range(n)]
    prompts[0] = 77
    s.check(prompts, s.append(prompts))
    s.fork([0] * (n // 2) + [rng.randrange(n) for _ in range(n - n // 2)])
    s.check(None, None)
    for step in range(14):
        new = [0 if rng.random() < 0.1 else rng.choice([1, 1, 1, rng.randint(1, 20)]) for _ in range(n)]
        new = [min(a, width * page - len(h)) for a, h in zip(new, s.history)]
        new[0] = max(new[0], 1)
        got = s.append(new)
        assert not s.missing.any()
        s.check(new, got)
        if rng.random() < 0.7:
            s.fork([rng.choice([i, i, rng.randrange(n), -1 if rng.random() < 0.2 else i]) for i in range(n)])
        if rng.random() < 0.3 and not window:                    # drafted tokens that were refused, within the open page (behind a
            # window a shorter length would see positions that were given back)
            drop = [rng.randint(0, len(h) % page) for h in s.history]
            s.history = [h[:len(h) - d] for h, d in zip(s.history, drop)]
            s.lens -= ints(drop)
        if rng.random() < 0.5:
            s.release()
        if rng.random() < 0.4:
            s.compact()
        s.check(None, None)
        if not s.history[0]:
            s.append([5] + [0] * (n - 1))
    s.release(ints([0] * n))
    assert not s.refs.any() and (s.pages == -1).all()


@pytest.mark.parametrize("bits", [8, 16])
def test_tokens_dropped_into_a_shared_page(bits):
    """After a fork at a page's border one of the two goes back into the shared page and writes other tokens there."""
    import torch
    s = Server(2, 16, bits, 20, 5, seed=1)
    s.append([32, 0])
    s.fork([0, 0])
    s.history[1] = s.history[1][:27]
    s.lens.copy_(ints([32, 27]))
    got = s.append([1, 9])
    s.check([1, 9], got)
    s.history[0] = s.history[0][:20]                             # and the other one
    s.lens.copy_(ints([20, 36]))
    got = s.append([3, 1])
    s.check([3, 1], got)


@pytest.mark.parametrize("bits", [8, 16])
def test_pool_runs_out(bits):
    """Too few pages: who got none is told, keeps what it has, and nobody's rows are overwritten."""
    import torch
    s = Server(3, 16, bits, 5, 4, seed=2)
    s.append([40, 0, 0])                                         # three pages
    s.fork([0, 0, 0])
    new = [1, 1, 1]
    kv = s.rows(3)
    s.lens += ints(new)
    s.enqueue_append(kv, ints([0, 1, 2, 3]), 3, 1)
    assert s.missing.tolist() == [0, 0, 0]                       # the first keeps the shared page, the others take the last two
    s.fork([0, 0, 2])
    s.lens += ints(new)
    s.enqueue_append(s.rows(3), ints([0, 1, 2, 3]), 3, 1)
    assert s.missing.tolist() == [0, 0, 0]
    s.fork([0, 0, 0])
    s.lens += ints([8, 8, 8])                                    # into a page that is not there for all
    s.enqueue_append(s.rows(24), ints([0, 8, 16, 24]), 24, 8)
    assert s.missing.tolist() == [0, 1, 2]                       # two pages, in order: the first's new block, the second's shared one
    named = s.pages[s.pages >= 0]
    assert torch.equal(torch.bincount(named.long(), minlength=5), s.refs.long())
    sh = s.shape(s.caches[0], 3, 1)
    s.attend(sh, moe.kv_batch(ints([0, 1, 2, 3]), s.lens, s.pages, s.slots), s.caches[0], 3)


@pytest.mark.parametrize("bits", [8, 16])
def test_captured_step(bits):
    """Fork, pages, copies, append and attention of a step in one graph, replayed with other parents and rows; the same
    steps eagerly beside it, with the program's own work between the replays."""
    import torch
    n = 6
    a, b = (Server(n, 16, bits, 200, 12, 40, 4, seed=3) for _ in range(2))
    for s in (a, b):
        s.append([30, 17, 16, 1, 50, 9])
    starts, kv = ints(range(n + 1)), a.rows(n)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    saved = [t.clone() for t in (a.pages, a.refs, a.lens, a.slots)] + [t.clone() for t in a.caches[0].handle.tensors if t is not None]

    def step():
        a.enqueue_fork()
        a.lens.add_(1)
        return a.enqueue_append(kv, starts, n, 1)

    with torch.cuda.stream(stream):
        step()                                                   # everything is loaded before the capture
    torch.cuda.synchronize()
    for t, old in zip([a.pages, a.refs, a.lens, a.slots] + [t for t in a.caches[0].handle.tensors if t is not None], saved):
        t.copy_(old)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        out = step()
    rng = random.Random(5)
    for _ in range(40):
        parent = [rng.choice([i, rng.randrange(n)]) for i in range(n)]
        rows = b.rows(n)
        b.fork(parent)
        for s in range(n):
            b.history[s].append(rows[s])
        b.lens += 1
        want = b.enqueue_append(rows, starts, n, 1)
        a.parent.copy_(ints(parent))
        kv.copy_(rows)
        g.replay()
        torch.cuda.synchronize()
        for x, y in ((a.pages, b.pages), (a.refs, b.refs), (a.lens, b.lens), (out[0], want[0]), (out[1], want[1])):
            assert torch.equal(x, y)
    b.check([1] * n, want)


def test_other_stream():
    """The whole step on a stream of its own, the tables made on another."""
    import torch
    s = Server(4, 32, 8, 60, 8, 50, 4, seed=7)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        s.append([40, 3, 0, 90])
        s.fork([0, 3, 3, 0])
        got = s.append([1, 5, 1, 1])
    torch.cuda.synchronize()
    s.check([1, 5, 1, 1], got)
