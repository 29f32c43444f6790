"""Drafted tokens dropped again and again from an 8-bit cache: a page's rows stay in bf16 until a row of the page after the
next is appended, and every length whose open page still has its rows, or that has no open page, gives bit for bit what
the tokens that are left give when they are appended at once."""
import numpy as np
import pytest

import int4_routed_expert_02_amd as moe
from kv_testutil import Batch, poison
from test_gpu_kv_append import append, new_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.load()


class Tokens:
    """One sequence's tokens (rows of a pool) in a cache, and which pages' rows are gone by the header's rule."""

    def __init__(self, page, most, seed):
        self.P, self.rng, self.now, self.gone = page, np.random.RandomState(seed), [], set()
        self.b = Batch([most], [most], 2, 2, 64, bits=8, page=page, seed=seed)
        self.fresh = Batch([most], [most], 2, 2, 64, bits=8, page=page, seed=seed + 1)
        _, self.k, self.v = new_rows(self.b, seed=seed)
        poison(self.b.cache)

    def append(self, n):
        import torch
        ids = self.rng.randint(0, self.k.shape[0], n).tolist()
        start, self.now = len(self.now), self.now + ids
        at = torch.tensor(ids).cuda()
        append(self.b.sub([n], [len(self.now)]), self.k[at], self.v[at])
        newest = (len(self.now) - 1) // self.P
        self.gone -= {i for i in self.gone if i * self.P >= start}
        self.gone |= set(range(max(newest - 1, 0)))

    def may_drop_to(self, length):
        return length % self.P == 0 or length // self.P not in self.gone

    def drop_to(self, length):
        assert length <= len(self.now) and self.may_drop_to(length)
        self.now = self.now[:length]

    def check(self, tag):
        import torch
        n = len(self.now)
        if n == 0:
            return
        poison(self.fresh.cache)
        at = torch.tensor(self.now).cuda()
        whole = self.fresh.sub([n], [n])
        append(whole, self.k[at], self.v[at])
        for got, want in zip(self.b.sub([n], [n]).read(), whole.read()):
            assert torch.equal(got, want), tag


@pytest.mark.parametrize("page", [16, 64])
def test_drops_from_one_longest_length(page):
    """Several drops in a row, down to a page below the longest length; then to a page's start, and on from there."""
    t = Tokens(page, 6 * page, 3)
    longest = 2 * page + 2
    t.append(longest)
    for length in (2 * page, longest - page + 5, longest - page + 1, longest - page):
        t.drop_to(length)
        t.check(f"dropped to {length}")
    t.append(2)
    t.check("two more")
    t.drop_to(longest - page)                  # the longest length still counts
    t.check("dropped again")
    assert not t.may_drop_to(page - 1) and not t.may_drop_to(1)
    t.drop_to(page)
    t.check("a page's start")
    t.append(page // 2)
    t.append(2 * page)
    t.drop_to(len(t.now) - page)
    t.check("on from there")
    t.drop_to(0)
    t.append(3)
    t.check("from the beginning")


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("seed", [1, 2])
def test_walks(page, seed):
    """Appends of a few tokens or several pages, drops to any length that may be dropped to."""
    most = 6 * page
    t, rng = Tokens(page, most, seed), np.random.RandomState(seed + 50)
    drops = 0
    for step in range(60):
        n = len(t.now)
        to = int(rng.randint(max(0, n - 2 * page), n + 1)) if rng.rand() < 0.5 else n
        if to < n and t.may_drop_to(to):
            t.drop_to(to)
            drops += 1
        else:
            room = most - n
            if room == 0:
                t.drop_to(most - page)
            else:
                t.append(min(room, int(rng.randint(1, 9)) if rng.rand() < 0.6 else int(rng.randint(1, 3 * page))))
        t.check(f"step {step}: {n} tokens to {len(t.now)}")
    assert drops >= 5
