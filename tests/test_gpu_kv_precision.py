"""moe_kv_attention's f32 outputs and log-sum-exp against 64 bits under the bound that the stated precision gives.

A weight enters the product with the values as two bf16 parts, off by at most 2^-16 of itself.  Its exponent comes from an
f32 score, off by (D / 8 + 8) * 2^-24 * sum |scale q k|, scaled, shifted by the maximum and joined with the value scale's
logarithm in at most 8 roundings of numbers no larger than that sum and 16; the exponential itself is good to 2^-22.  An
output's sum over n positions passes one product instruction of 6 roundings for every 16 of them and at most 128 more in
rescaling and joining, all relative to sum w |v|."""
import numpy as np
import pytest

import int4_routed_expert_02_amd as moe
import kv_testutil
from gpu_util import say
from kv_testutil import Batch, attention64, fill
from test_gpu_kv_attention import attend, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.load()


def one_part(w):
    """Weights rounded to a single bf16 value (nearest, ties to even)."""
    b = w.astype(np.float32).view(np.uint32)
    return ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32).astype(np.float64)


def rounded_weights64(b, q):
    """The outputs that weights of one bf16 value would give."""
    out, G, qn = np.zeros((b.rows, b.Hq, b.D)), b.Hq // b.H, kv_testutil.bf16_np(q)
    for s in range(len(b.new)):
        k, v, present = kv_testutil.stored(b, s)
        for i in range(b.new[s]):
            p, row = b.lens[s] - b.new[s] + i, int(b.row_start[s]) + i
            for h in range(b.Hq):
                z = k[:p + 1, h // G] @ qn[row, h] * b.scale
                w = np.exp(z - z.max())
                out[row, h] = one_part(w) @ v[:p + 1, h // G] / w.sum()
    return out


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("heads", [(8, 2, 64), (8, 2, 128), (4, 4, 64)], ids=lambda h: "-".join(map(str, h)))
@pytest.mark.parametrize("new,lens", [([1, 1, 3, 1], [5, 70, 33, 300]), ([40, 70], [40, 200])], ids=["few", "many"])
def test_stated_precision(new, lens, heads, bits):
    b = Batch(new, lens, *heads, bits=bits, page=16, seed=51)
    fill(b)
    q = queries(b, std=0.5)
    ref, mag, ref_lse, zmag = attention64(b, q)
    n = np.concatenate([np.arange(l - m, l) + 1 for m, l in zip(new, lens)])[:, None]
    z_tol = (b.D / 8 + 8) * 2.0 ** -24 * zmag + 8 * 2.0 ** -24 * (zmag + 16)
    tol = mag * (2.0 ** -16 + 2.0 ** -22 + z_tol + (6 * n / 16 + 128) * 2.0 ** -24)[..., None]
    tol = np.maximum(tol, 1e-30)                 # a code of 0 at a row's only position
    out, lse = (t.double().cpu().numpy() for t in attend(b, q))
    err = np.abs(out - ref) / tol
    lerr = np.abs(lse - ref_lse) / (z_tol + 2.0 ** -22 + (n + 128) * 2.0 ** -24)
    worse = np.abs(rounded_weights64(b, q) - ref) / tol
    say(f"precision {heads} new {new} {bits} bits: out {err.max():.3f} of the bound, lse {lerr.max():.3f}; one bf16 value a weight {worse.max():.1f}")
    assert (err <= 1).all() and (lerr <= 1).all()
    assert worse.max() > 4                       # the bound tells the two apart
