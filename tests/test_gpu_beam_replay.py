"""What the beam-search example returns, taken apart: every returned sequence is run again as one of a batch that forks nothing,
with its tokens given, and the log-probabilities of these tokens, in 64 bits from the logits of that run, have to add up to the
returned score.  A wrong parent, slot, page or last row, or tokens of another beam, give other sums.

The search and the replay run the same calls with the same numbers of rows and sequences, and no operation of the layers mixes
tokens, so the logits are the same numbers and only the scores' roundings are left: every step rounds the sum once to f32, half
a step, 2^-24 of it; both sides' sums in 64 bits are nearer than that by far."""
import os
import sys

import numpy as np
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
    return [[(11 * i * i + 5 * i + 71 * r) % vocab for i in range(90 - 37 * r)] for r in range(n)]


def replay(ex, n_layers, requests, beams, texts, tokens, vocab, seed=0):
    """Log-probabilities [requests][steps][vocab] (64 bits) before every token of tokens [requests][steps], which are
    sequence `request * beams` of a batch; the others hold token 0."""
    import torch
    dl, steps = ex.dl, tokens.shape[1]
    longest = max(map(len, texts))
    state = ex.Beams(requests, beams, longest + steps)
    layers = dl.stack(n_layers, state, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    width = layers[0].norms[0].numel()
    embed = torch.randn(vocab, width, generator=gen, device="cuda").to(torch.bfloat16)
    head, norm = dl.linear_weights(vocab, width, gen), torch.rand(width, generator=gen, device="cuda") + 0.5
    cos, sin = dl.tables(longest + steps)

    def forward(ids, new):
        batch, sizes = state.rows(layers, new)
        x = embed[ids]
        for layer in layers:
            x = layer.forward(x, batch, sizes, cos, sin)
        return x

    x = forward(torch.tensor([t for p in texts for t in p], device="cuda"),
                [len(texts[s // beams]) if s % beams == 0 else 0 for s in range(state.n_seq)])
    last = torch.zeros(state.n_seq, width, dtype=torch.bfloat16, device="cuda")
    last[::beams] = x[torch.tensor(np.cumsum([len(p) for p in texts]) - 1, device="cuda")]
    out = []
    for step in range(steps):
        logits = dl.DecoderLayer.linear(dl.rms_norm(last, norm), head)[::beams]
        out.append(logits.double().log_softmax(1))
        ids = torch.zeros(state.n_seq, dtype=torch.long, device="cuda")
        ids[::beams] = tokens[:, step].long()
        if step + 1 < steps:
            last = forward(ids, [1] * state.n_seq)
    assert not state.missing.any()
    return torch.stack(out, 1)


@pytest.mark.parametrize("requests,beams,steps,vocab,end", [(2, 4, 9, 2001, -1), (3, 3, 7, 700, 5), (1, 6, 5, 40, 3), (2, 1, 8, 1000, -1)])
def test_scores_are_the_sequences_own(ex, requests, beams, steps, vocab, end):
    import torch
    texts = prompts(requests, vocab)
    tokens, scores, _ = ex.search(2, requests, beams, texts, steps, vocab, end_token=end, compact=steps % 2 == 1)
    assert int(tokens.min()) >= 0 and int(tokens.max()) < vocab
    seen = set()
    for b in range(beams):
        logp = replay(ex, 2, requests, beams, texts, tokens[:, b], vocab)
        own = logp.gather(2, tokens[:, b].long()[..., None])[..., 0]
        if end >= 0:                                             # behind its end a beam stands still
            ended = ((tokens[:, b] == end).int().cumsum(1) - (tokens[:, b] == end).int()) > 0
            assert (tokens[:, b][ended] == end).all()
            own = torch.where(ended, 0.0, own)
        got, want = scores[:, b].double(), own.sum(1)
        assert ((got - want).abs() <= steps * (2.0 ** -24 * want.abs() + 2.0 ** -38)).all(), (got, want)
        for r in range(requests):
            assert (r, tuple(tokens[r, b].tolist())) not in seen
            seen.add((r, tuple(tokens[r, b].tolist())))
        if beams == 1:                                           # greedy: the largest logit each time, of equal ones the first
            assert torch.equal(logp.argmax(2), tokens[:, b].long())


def test_best_of_all(ex):
    """As many beams as there are sequences: the search has to return all of them in order, against every one run for itself."""
    import itertools
    import torch
    vocab, steps, texts = 5, 3, prompts(1, 5)
    tokens, scores, _ = ex.search(1, 1, 125, texts, steps, vocab)
    every = torch.tensor(list(itertools.product(range(vocab), repeat=steps)), device="cuda")
    sums = []
    for seq in every:
        logp = replay(ex, 1, 1, 125, texts, seq[None], vocab)
        sums.append(logp[0].gather(1, seq[:, None]).sum())
    sums = torch.stack(sums)
    assert sorted(map(tuple, tokens[0].tolist())) == sorted(map(tuple, every.tolist()))
    place = {tuple(t): i for i, t in enumerate(every.tolist())}
    want = sums[torch.tensor([place[tuple(t)] for t in tokens[0].tolist()], device="cuda")]
    assert ((scores[0].double() - want).abs() <= steps * (2.0 ** -24 * want.abs() + 2.0 ** -38)).all()
    assert (scores[0, :-1] >= scores[0, 1:]).all()
