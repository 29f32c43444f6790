"""Beam search on the library's calls: the layers of decoder_layer.py, an output head, and the beams' pages on the device.

    python examples/beam_search.py [--layers 2] [--requests 2] [--beams 4] [--prompt 100] [--steps 12]

Two prompts are read into one beam each; every step then takes the best continuations (moe_beam_select), lets the beams
follow their parents (moe_kv_fork and, for the open pages, moe_kv_copy), hands out pages for the next token
(moe_kv_reserve) and runs the layers.  The tables stay on the device: the host knows lengths alone, and reads the tokens
once, at the end.  Random weights, so the text says nothing.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import numpy as np  # noqa: E402
import torch  # noqa: E402

import decoder_layer as dl  # noqa: E402
import int4_routed_expert_02_amd as moe  # noqa: E402


def ints(*shape, fill=-1):
    return torch.full(shape, fill, dtype=torch.int32, device="cuda")


class Beams:
    """The state of requests * beams sequences: page tables over one pool, which every layer's cache is laid out by."""

    def __init__(self, requests, beams, max_len):
        self.requests, self.beams, self.n_seq = requests, beams, requests * beams
        self.max_pages = -(-max_len // dl.PAGE)
        self.n_pages = self.n_seq * (self.max_pages + 1)          # as if no page were shared: the pool cannot run out
        self.pages, self.next_pages = ints(self.n_seq, self.max_pages), ints(self.n_seq, self.max_pages)
        self.refs = ints(self.n_pages, fill=0)
        self.kv_len, self.next_len = ints(self.n_seq, fill=0), ints(self.n_seq, fill=0)
        self.slots, self.next_slots = torch.arange(self.n_seq, dtype=torch.int32, device="cuda"), ints(self.n_seq)
        self.slot_src, self.slot_dst, self.missing = ints(self.n_seq), ints(self.n_seq), ints(self.n_seq)
        self.moves = ints(2, self.n_pages // 2)
        self.longest = 0

    def sizes(self, rows=0, max_rows=0):
        return dict(n_seq=self.n_seq, rows=rows, max_rows=max_rows, max_len=self.longest, q_heads=dl.Q_HEADS, max_pages=self.max_pages)

    def workspace(self, sh):
        return torch.empty(moe.moe_kv_pool_workspace_bytes(sh), dtype=torch.uint8, device="cuda")

    def rows(self, layers, new):
        """Pages for `new[s]` more tokens of each sequence: the batch's tables and sizes."""
        starts = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).cuda()
        self.kv_len += torch.tensor(new, dtype=torch.int32, device="cuda")
        self.longest += max(new)
        batch, sizes = moe.kv_batch(starts, self.kv_len, self.pages, self.slots), self.sizes(sum(new), max(new))
        sh = layers[0].cache.shape(**sizes)
        moe.moe_kv_reserve(sh, batch, self.pages, self.refs, missing=self.missing, ws=self.workspace(sh))
        return batch, sizes

    def follow(self, layers, parent):
        """Every sequence goes on from its parent: shared pages, and copies of the pages still being written."""
        sh = layers[0].cache.shape(**self.sizes())
        before = moe.kv_batch(ints(self.n_seq + 1, fill=0), self.kv_len, self.pages, self.slots)
        moe.moe_kv_fork(sh, before, parent, self.next_len, self.next_pages, self.next_slots, self.refs, self.slot_src, self.slot_dst)
        self.kv_len, self.next_len = self.next_len, self.kv_len
        self.pages, self.next_pages = self.next_pages, self.pages
        self.slots, self.next_slots = self.next_slots, self.slots
        for layer in layers:
            moe.moe_kv_copy(sh, layer.cache.handle, slot_src=self.slot_src, slot_dst=self.slot_dst)

    def compact(self, layers):
        """The pages in use to the front of every layer's cache."""
        sh = layers[0].cache.shape(**self.sizes())
        moe.moe_kv_compact(sh, self.pages, self.refs, *self.moves, ws=self.workspace(sh))
        for layer in layers:
            moe.moe_kv_copy(sh, layer.cache.handle, page_src=self.moves[0], page_dst=self.moves[1])


def search(n_layers, requests, beams, prompts, steps, vocab, end_token=-1, seed=0, compact=False):
    """tokens [requests][beams][steps] and scores [requests][beams] of the best beams for the prompts' token ids; compact:
    move the pages together after every step."""
    state = Beams(requests, beams, max(map(len, prompts)) + steps)
    layers = dl.stack(n_layers, state, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    width = layers[0].norms[0].numel()
    embed = torch.randn(vocab, width, generator=gen, device="cuda").to(torch.bfloat16)
    head, norm = dl.linear_weights(vocab, width, gen), torch.rand(width, generator=gen, device="cuda") + 0.5
    cos, sin = dl.tables(max(map(len, prompts)) + steps)

    def forward(tokens, new):
        batch, sizes = state.rows(layers, new)
        x = embed[tokens]
        for layer in layers:
            x = layer.forward(x, batch, sizes, cos, sin)
        return x

    new = [len(prompts[s // beams]) if s % beams == 0 else 0 for s in range(state.n_seq)]
    x = forward(torch.tensor([t for p in prompts for t in p], device="cuda"), new)
    last = torch.zeros(state.n_seq, width, dtype=torch.bfloat16, device="cuda")
    last[::beams] = x[torch.tensor(np.cumsum([len(p) for p in prompts]) - 1, device="cuda")]
    scores = torch.full((requests, beams), -float("inf"), device="cuda")
    scores[:, 0] = 0.0                                           # one beam is alive
    done = torch.zeros(requests, beams, dtype=torch.bool, device="cuda") if end_token >= 0 else None
    ws = torch.empty(moe.moe_beam_workspace_bytes(requests, beams, vocab, beams), dtype=torch.uint8, device="cuda")
    history = []
    for step in range(steps):
        logits = dl.DecoderLayer.linear(dl.rms_norm(last, norm), head)
        parent, token, score = ints(requests, beams), ints(requests, beams), torch.empty_like(scores)
        ended = torch.empty_like(done) if done is not None else None
        moe.moe_beam_select(logits, scores, parent, token, score, done=done, done_out=ended, end_token=end_token, ws=ws)
        history.append((parent, token))
        scores, done = score, ended
        if step + 1 < steps:
            state.follow(layers, parent.flatten())
            if compact:
                state.compact(layers)
            last = forward(token.flatten().clamp(min=0), [1] * state.n_seq)
    # the tokens from the last step back
    row, out = torch.arange(state.n_seq, device="cuda"), []
    for parent, token in reversed(history):
        out.append(token.flatten()[row])
        row = parent.flatten()[row].long()
    return torch.stack(out[::-1], 1).view(requests, beams, steps), scores, state


def main():
    ap = argparse.ArgumentParser()
    for name, value in (("layers", 2), ("requests", 2), ("beams", 4), ("prompt", 100), ("steps", 12), ("vocab", 5003)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    rs = np.random.RandomState(0)
    prompts = [rs.randint(0, a.vocab, max(1, a.prompt - 17 * r)).tolist() for r in range(a.requests)]
    tokens, scores, state = search(a.layers, a.requests, a.beams, prompts, a.steps, a.vocab)
    alone = sum(-(-(len(p) + a.steps - 1) // dl.PAGE) for p in prompts) * a.beams
    print(f"{a.beams} beams of {a.requests} requests: {int((state.refs > 0).sum())} pages in use, {alone} if none were shared")
    for r in range(a.requests):
        for b in range(a.beams):
            print(f"request {r}, score {scores[r, b]:.4f}: {tokens[r, b].tolist()}")


if __name__ == "__main__":
    main()
