"""The decoder-layer example: its attention block against the same block in 64 bits, and the same tokens in other cuts.

Tolerances: the block's bf16 roundings are those of the norm's output, q/k/v, the rotated q and k, the attention output and
the sum with the residual, each 2^-8 relative at most; keys and values of full pages are off by half a code, 1 / 254 of
their page's largest.  Measured against the block's own update (without the residual), five roundings of 2^-8 and the codes
(about 3.5 / 254 of an rms each) give at most 3 percent of its rms in the 2-norm."""
import os
import sys

import pytest

import int4_routed_expert_02_amd as moe
from gpu_util import say

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.load()
    import decoder_layer
    return decoder_layer


def dequantised(weights):
    import torch
    codes, scales = weights
    b = codes.to(torch.int64)
    c = torch.stack((b & 15, b >> 4), dim=2).flatten(1)
    c = torch.where(c > 7, c - 16, c).double()
    return (c.unflatten(1, (scales.shape[1], -1)) * scales.double()[:, :, None]).flatten(1)


def attention_block64(ex, layer, x, cos, sin):
    """One sequence from position 0, in 64 bits: the block's update of x."""
    import torch
    n = x.shape[0]

    def norm(t, w):
        return t / (t.square().mean(-1, keepdim=True) + ex.EPS).sqrt() * w.double()

    h = norm(x.double(), layer.norms[0])
    qkv = (h @ dequantised(layer.qkv).T).unflatten(1, (-1, ex.DIM))
    q, k, v = qkv.split([ex.Q_HEADS, ex.KV_HEADS, ex.KV_HEADS], dim=1)
    c, s = cos[:n].double()[:, None], sin[:n].double()[:, None]

    def rotate(t):
        a, b = t.chunk(2, dim=-1)
        return torch.cat((a * c - b * s, a * s + b * c), dim=-1)

    q, k = rotate(norm(q, layer.q_norm)), rotate(norm(k, layer.k_norm))
    group = ex.Q_HEADS // ex.KV_HEADS
    k, v = k.repeat_interleave(group, 1).transpose(0, 1), v.repeat_interleave(group, 1).transpose(0, 1)
    z = q.transpose(0, 1) @ k.transpose(1, 2) / ex.DIM ** 0.5
    z = z.masked_fill(torch.ones(n, n, device=z.device).triu(1).bool(), -float("inf"))
    out = (z.softmax(-1) @ v).transpose(0, 1).flatten(1)
    return out @ dequantised(layer.out).T


def test_attention_block(ex):
    import torch
    seqs = ex.Sequences(1, 200)
    layer = ex.stack(1, seqs)[0]
    cos, sin = ex.tables(200)
    x = torch.randn(200, 1024, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(torch.bfloat16)
    batch, sizes = seqs.append([200])
    got = layer.attention(x, batch, sizes, cos, sin)
    ref = attention_block64(ex, layer, x, cos, sin)
    err = ((got.double() - x.double()) - ref).norm() / ref.norm()
    say(f"attention block: {float(err):.4f} of its update")
    assert err < 0.03


def test_cuts_agree(ex):
    """A prompt at once, and the same tokens in a chunk and single steps: the cache holds the same bits after the first
    layer's append, and the outputs agree to the roundings that the different kernels make."""
    import torch
    total, cuts = 150, [100, 37] + [1] * 13
    x = torch.randn(2 * total, 1024, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").to(torch.bfloat16)
    cos, sin = ex.tables(total)
    results = []
    for cut in ([total], cuts):
        seqs = ex.Sequences(2, total)
        layers = ex.stack(1, seqs)
        out, at = torch.empty_like(x), 0
        for n in cut:
            rows = torch.cat([torch.arange(at, at + n), torch.arange(total + at, total + at + n)]).cuda()
            batch, sizes = seqs.append([n, n])
            out[rows] = layers[0].attention(x[rows], batch, sizes, cos, sin)
            at += n
        results.append((out, layers[0].cache))
    (a, ca), (b, cb) = results
    full = torch.cat([seqs.pages[s, :total // ex.PAGE] for s in range(2)]).long()
    for name in ("k", "v", "k_scale", "v_scale"):
        u, w = getattr(ca, name)[full], getattr(cb, name)[full]
        same = (u == w).float().mean().item()
        say(f"cuts: {name} equal in {same:.6f}")
        assert same > 0.99        # a projection's sums run in another order for another number of rows
    err = (a.double() - b.double()).norm() / (a.double() - x.double()).norm()
    say(f"cuts: outputs differ by {float(err):.4f} of the update")
    assert err < 0.03


def test_example_runs(ex, capsys, monkeypatch):
    monkeypatch.setattr(sys, "argv", ["decoder_layer.py", "--layers", "2", "--prompt", "130", "--steps", "3"])
    ex.main()
    out = capsys.readouterr().out
    assert "decode step 2: lengths [133, 68]" in out and "nan" not in out
