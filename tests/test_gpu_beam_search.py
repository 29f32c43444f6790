"""The beam-search example: that it runs, that its result does not depend on which pages hold what (bit for bit), that its
scores are in order and that one beam is the greedy choice."""
import os
import sys

import pytest

import int4_routed_expert_02_amd as moe

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.load()
    import beam_search
    return beam_search


def prompts(n, vocab):
    return [[(7 * i * i + 31 * r) % vocab for i in range(130 - 41 * r)] for r in range(n)]


def test_pages_do_not_matter(ex):
    """The pages moved together after every step, and left where they are: the same tokens and scores, bit for bit."""
    import torch
    results = [ex.search(2, 2, 4, prompts(2, 3001), 10, 3001, end_token=5, compact=c) for c in (False, True)]
    (t0, s0, a), (t1, s1, b) = results
    assert torch.equal(t0, t1) and torch.equal(s0.view(torch.int32), s1.view(torch.int32))
    for state in (a, b):
        named = state.pages[state.pages >= 0]
        assert torch.equal(torch.bincount(named.long(), minlength=state.n_pages), state.refs.long())
        assert not state.missing.any()
    live = int((b.refs > 0).sum())
    assert (b.refs[live + b.n_seq:] == 0).all()                  # in front, but for the last step's new pages
    assert int((a.refs > 0).sum()) < 2 * 4 * 3                   # the prompts' full pages are shared
    assert (s0[:, :-1] >= s0[:, 1:]).all() and (s0 < 0).all()


def test_one_beam_is_greedy(ex):
    """A single beam takes the largest logit of every step; the first tokens of several beams come from one distribution."""
    import torch
    t1, s1, _ = ex.search(1, 2, 1, prompts(2, 1000), 6, 1000)
    t8, s8, _ = ex.search(1, 2, 8, prompts(2, 1000), 1, 1000)
    assert torch.equal(t1[:, 0, 0], t8[:, 0, 0])
    assert len(set(t8[0, :, 0].tolist())) == 8 and len(set(t8[1, :, 0].tolist())) == 8
    assert (s1 < s8[:, :1]).all()


def test_example_runs(ex, capsys, monkeypatch):
    monkeypatch.setattr(sys, "argv", ["beam_search.py", "--layers", "1", "--prompt", "70", "--steps", "5"])
    ex.main()
    out = capsys.readouterr().out
    assert "4 beams of 2 requests" in out and out.count("score") == 8 and "nan" not in out
