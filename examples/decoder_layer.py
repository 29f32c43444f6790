"""A whole decoder layer on the library's calls: int4 projections, the paged 8-bit cache, attention and the MoE layer.

    python examples/decoder_layer.py [--layers 2] [--prompt 300] [--steps 8]

Runs a stack of Nano-shaped layers (width 1024, 16 query and 4 key/value heads of 64 with per-head norms, 64 experts top-2
and a shared expert, random weights) over two sequences: their prompts in one call, then a few decode steps, and prints the
time of a step.  torch holds the tensors, norms the layer inputs and adds the residuals; everything else runs in the
library.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import numpy as np  # noqa: E402
import torch  # noqa: E402

import int4_routed_expert_02_amd as moe  # noqa: E402

Q_HEADS, KV_HEADS, DIM, GROUP, PAGE, EPS = 16, 4, 64, 64, 64, 1e-6


def rms_norm(x, weight):
    f = x.float()
    return (f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * weight).to(torch.bfloat16)


def linear_weights(n, k, gen):
    """Random [n][k] weights as packed int4 codes with one scale for every GROUP of k."""
    w = torch.randn(n, k, generator=gen, device="cuda") * k ** -0.5
    codes, scales = moe.moe_quantize_rows(w.view(-1, GROUP), 4)
    return codes.view(n, k // 2), scales.view(n, k // GROUP)


class Sequences:
    """The batch's tables: which pages each sequence has, how long it is, which rows of a call are its own."""

    def __init__(self, n_seq, max_len):
        self.n_seq, self.max_pages = n_seq, -(-max_len // PAGE)
        self.n_pages = n_seq * self.max_pages
        self.lens = [0] * n_seq
        order = np.random.RandomState(0).permutation(self.n_pages).astype(np.int32)
        self.pages = torch.from_numpy(order.reshape(n_seq, self.max_pages)).cuda()

    def append(self, new):
        """Rows for `new[s]` more tokens of each sequence: the batch's tables and sizes."""
        self.lens = [a + b for a, b in zip(self.lens, new)]
        starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        batch = moe.kv_batch(torch.from_numpy(starts).cuda(), torch.tensor(self.lens, dtype=torch.int32, device="cuda"), self.pages)
        sizes = dict(n_seq=self.n_seq, rows=int(starts[-1]), max_rows=max(new), max_len=max(self.lens), q_heads=Q_HEADS,
                     max_pages=self.max_pages)
        return batch, sizes


class DecoderLayer:
    def __init__(self, cfg, moe_arrays, seqs: Sequences, gen):
        H = cfg.H
        self.qkv = linear_weights((Q_HEADS + 2 * KV_HEADS) * DIM, H, gen)
        self.out = linear_weights(H, Q_HEADS * DIM, gen)
        self.norms = [torch.rand(H, generator=gen, device="cuda") + 0.5 for _ in range(2)]
        self.q_norm, self.k_norm = (torch.rand(DIM, generator=gen, device="cuda") + 0.5 for _ in range(2))
        self.cache = moe.KvPages(seqs.n_pages, KV_HEADS, DIM, PAGE, 8, seqs.n_seq)
        self.moe = moe.MoeLayer(cfg, moe_arrays)

    @staticmethod
    def linear(x, weights, residual=None):
        out = torch.empty(x.shape[0], weights[0].shape[0], dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(moe.moe_linear_q4_workspace_bytes(*out.shape, x.shape[1]), dtype=torch.uint8, device="cuda")
        moe.moe_linear_q4(x, *weights, out, residual, ws)
        return out

    def attention(self, x, batch, sizes, cos, sin):
        """x plus the attention block's output; the rows' keys and values go into the cache."""
        rows = x.shape[0]
        qkv = self.linear(rms_norm(x, self.norms[0]), self.qkv)
        q, k, v = (t.unflatten(1, (-1, DIM)) for t in qkv.split([Q_HEADS * DIM, KV_HEADS * DIM, KV_HEADS * DIM], dim=1))
        sh = self.cache.shape(**sizes)
        rot = moe.kv_rotary(cos, sin, DIM, None, self.q_norm, self.k_norm, EPS)
        rotated, seen = (torch.empty(rows, Q_HEADS, DIM, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        moe.moe_kv_append(sh, batch, self.cache.handle, k, v, rot, q, rotated)
        ws = torch.empty(moe.moe_kv_workspace_bytes(sh), dtype=torch.uint8, device="cuda")
        moe.moe_kv_attention(sh, batch, self.cache.handle, rotated, seen, None, ws)
        return self.linear(seen.flatten(1), self.out, residual=x)

    def forward(self, x, batch, sizes, cos, sin):
        x = self.attention(x, batch, sizes, cos, sin)
        h = rms_norm(x, self.norms[1])
        y = torch.empty_like(x)
        self.moe.forward(h, y, self.moe.workspace(x.shape[0]))
        return x + y


def tables(n_pos):
    """cos and sin of position times frequency, [n_pos][DIM / 2]."""
    half = DIM // 2
    angle = torch.arange(n_pos, device="cuda", dtype=torch.float64)[:, None] * \
        10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    return angle.cos().float(), angle.sin().float()


def stack(n_layers, seqs, seed=0):
    import synth
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    cfg = synth.CONFIGS["c0"]
    return [DecoderLayer(cfg, synth.layer(cfg.with_(seed=cfg.seed + i)), seqs, gen) for i in range(n_layers)]


def run(layers, seqs, x, new, cos, sin):
    """The rows x of all sequences, `new[s]` of each, through the layers."""
    batch, sizes = seqs.append(new)
    for layer in layers:
        x = layer.forward(x, batch, sizes, cos, sin)
    return x


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    seqs = Sequences(2, a.prompt + a.steps)
    layers = stack(a.layers, seqs)
    cos, sin = tables(a.prompt + a.steps)
    new = [a.prompt, max(1, a.prompt // 2)]
    x = torch.randn(sum(new), layers[0].norms[0].numel(), device="cuda").to(torch.bfloat16)
    y = run(layers, seqs, x, new, cos, sin)
    print(f"prompts of {new} tokens through {a.layers} layers: output rms {y.float().square().mean().sqrt().item():.3f}")
    last = y[torch.tensor([new[0] - 1, sum(new) - 1], device="cuda")]
    for step in range(a.steps):
        torch.cuda.synchronize()
        t = time.perf_counter()
        last = run(layers, seqs, last, [1, 1], cos, sin)
        torch.cuda.synchronize()
        print(f"decode step {step}: lengths {seqs.lens}, {1e6 * (time.perf_counter() - t):.0f} us, "
              f"output rms {last.float().square().mean().sqrt().item():.3f}")


if __name__ == "__main__":
    main()
