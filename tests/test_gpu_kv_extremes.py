"""moe_kv_attention with scores and values far from one: scores whose f32 spacing is many units leave one position with the
weight 1, and the row gets that position's value and score, wherever the scores lie.

A score is off by at most (D / 8 + 8) * 2^-24 * sum |scale q k| (f32 sums of exact products, in tiles), so where the best
leads the second by more than twice that and 60 the others' weights are below 2^-80.  The value then passes one product
with a weight of two bf16 parts (2^-16) and a few f32 roundings."""
import numpy as np
import pytest

import int4_routed_expert_02_amd as moe
from gpu_util import say
from kv_testutil import Batch, bf16_np, fill, stored
from test_gpu_kv_attention import attend, check, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.load()


def check_best(b, q, tag, most_unclear=0.1):
    """Rows with a clear best position have its value and score."""
    out, lse = (t.double().cpu().numpy() for t in attend(b, q))
    qn, G, clear, unclear, worst = bf16_np(q), b.Hq // b.H, 0, 0, 0.0
    for s in range(len(b.new)):
        k, v, present = stored(b, s)
        for i in range(b.new[s]):
            p, row = b.lens[s] - b.new[s] + i, int(b.row_start[s]) + i
            seen = np.nonzero(present[:p + 1])[0]
            for h in range(b.Hq):
                kk, vv = k[seen, h // G], v[seen, h // G]
                z, tol = kk @ qn[row, h] * b.scale, (b.D / 8 + 8) * 2.0 ** -24 * (np.abs(kk) @ np.abs(qn[row, h])).max() * abs(b.scale)
                best = int(z.argmax())
                rest = np.delete(z, best)
                assert np.isfinite(out[row, h]).all() and np.isfinite(lse[row, h]), (tag, row, h)
                if rest.size and z[best] - rest.max() < 2 * tol + 60:
                    unclear += 1
                    continue
                clear += 1
                err = np.abs(out[row, h] - vv[best]) / (2.0 ** -15 * np.abs(vv[best]) + 1e-30)
                worst = max(worst, err.max())
                assert (err <= 1).all(), (tag, row, h, err.max())
                assert abs(lse[row, h] - z[best]) <= tol + 4 * 2.0 ** -24 * abs(z[best]) + 1e-5, (tag, row, h)
    say(f"{tag}: {clear} rows and heads with a clear best, {unclear} without, {worst:.3f} of the bound")
    assert unclear <= most_unclear * (clear + unclear)


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("dim,size", [(64, 1e12), (64, 1e16), (128, 1e18)])
@pytest.mark.parametrize("new,lens", [([1, 1, 1, 1], [1, 2, 20, 45]), ([40, 1, 20], [40, 2, 33])], ids=["few", "many"])
def test_scores_far_below_zero(new, lens, dim, size, bits):
    """Every score of a row is a large negative number."""
    b = Batch(new, lens, 8, 2, dim, bits=bits, page=16, seed=31)
    fill(b, k_std=size)
    b.cache.k.abs_()
    if bits == 8:
        b.cache.k_tail.abs_()
    check_best(b, -queries(b).abs() * size, f"scores about -{size * size * dim ** 0.5:.0e}, new {new}, {bits} bits")


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("dim,size", [(64, 3e3), (64, 1e5), (64, 1e12), (128, 1e9), (128, 1e18)])
@pytest.mark.parametrize("new,lens", [([1, 1, 3], [300, 65, 700]), ([150, 40], [400, 300])], ids=["few", "many"])
def test_scores_whose_spacing_is_large(new, lens, dim, size, bits):
    """Tiles of 64 positions that every row sees, with scores from 1e8 to 1e37 of both signs."""
    b = Batch(new, lens, 8, 2, dim, bits=bits, page=32, seed=32)
    fill(b, k_std=size)
    check_best(b, queries(b) * size, f"scores about {size * size * dim ** 0.5:.0e}, new {new}, {bits} bits")


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("seqs,new", [(64, 1), (64, 4), (2, 130)], ids=["few", "several", "many"])
def test_values_near_the_largest_number(seqs, new, bits):
    """Every 512 positions the largest score grows by 5, all values are 2e38: the weights' sum is 1.007 times the largest,
    so nothing passes f32's range as long as no weight passes 1."""
    import torch
    length, dim, heads = 1600, 64, 8
    b = Batch([length] * seqs, [length] * seqs, heads, heads, dim, bits=bits, page=64, seed=33)
    z = np.full(length, -100.0)
    z[5::512] = 5.0 * np.arange(len(z[5::512]))
    k = torch.from_numpy(z / 8).to(torch.bfloat16).cuda()[None, :, None, None].expand(seqs, length, heads, dim).reshape(-1, heads, dim)
    v = torch.full_like(k, 2e38)
    moe.moe_kv_append(b.sh, b.batch, b.cache.handle, k.contiguous(), v)
    c = b.sub([new] * seqs, [length] * seqs)
    q = torch.ones(c.rows, heads, dim, dtype=torch.bfloat16, device="cuda")
    held = stored(b, 0)[0][:, 0, 0] * 8                                            # the scores that the cache's keys give
    best = torch.from_numpy(np.maximum.accumulate(held)[-new:]).cuda().repeat(seqs)   # the largest that each row sees
    for f32 in (True, False):
        out, lse = attend(c, q, f32=f32)
        assert ((out.double() / 2e38 - 1).abs() <= 2 ** -7).all(), out.flatten()[:4]
        assert ((lse - best[:, None]).abs() < 0.2).all()


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("new,lens", [([6, 1], [3, 200]), ([90, 40], [70, 40])], ids=["few", "many"])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 30, 2 ** 30])
def test_window_wider_than_any_sequence(window, new, lens, bits):
    """It hides nothing, from rows before position 0 either (they see the whole sequence where nothing is causal)."""
    b = Batch(new, lens, 4, 2, 64, bits=bits, page=16, window=window, flags=moe.MOE_KV_NONCAUSAL, seed=34)
    fill(b)
    check(b, queries(b), f"window {window}, new {new} of {lens}, {bits} bits")
