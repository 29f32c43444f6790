"""The header's rule for dropping tokens from an 8-bit cache, on a model of the open pages: row p of a sequence is kept in
half (p / P) % 2 at p % P, an append keeps the rows of its two newest pages."""
import random

import pytest


class OpenPages:
    def __init__(self, page):
        self.P, self.half, self.tokens, self.next = page, {}, [], 0

    def append(self, n):
        start = len(self.tokens)
        self.tokens += range(self.next, self.next + n)
        self.next += n
        newest = (len(self.tokens) - 1) // self.P
        for p in range(start, len(self.tokens)):
            if p // self.P >= newest - 1:
                self.half[p // self.P % 2, p % self.P] = self.tokens[p]

    def right(self, length):
        """Whether the rows of the page that this length leaves open are the tokens' own."""
        page = length // self.P
        return all(self.half.get((page % 2, p % self.P)) == self.tokens[p] for p in range(page * self.P, length))


@pytest.mark.parametrize("page", [4, 16])
@pytest.mark.parametrize("seed", range(20))
def test_lengths_from_the_longest_less_a_page_are_right(page, seed):
    rng, o, longest = random.Random(seed), OpenPages(page), 0
    for _ in range(60):
        n = rng.choice((1, 2, 5, page, 3 * page + 1))
        o.append(n)
        longest = max(longest, len(o.tokens))
        for length in range(len(o.tokens) + 1):
            if length >= longest - page or length % page == 0:
                assert o.right(length), (longest, length)
        o.tokens = o.tokens[:rng.randint(min(len(o.tokens), max(0, longest - page)), len(o.tokens))]


def test_a_page_from_the_present_length_is_too_much():
    """130 tokens in pages of 64, a page dropped and another one token later: page 0's first rows are those of page 2."""
    o = OpenPages(64)
    o.append(130)
    assert o.right(66)
    o.tokens = o.tokens[:66]
    o.append(1)
    assert not o.right(len(o.tokens) - 64) and o.right(64) and o.right(0)
