"""moe_linear_q4 where its offset is largest beside the result: few codes that are not 0, activations far from mean 0.

The bound is that of the f32 sums as derived in tests/test_gpu_linear_q4_extremes.py: a group's sum runs over x (c + 24) and
-24 x, so it is relative to 55 sum |x| of the group, whatever the codes are."""
import numpy as np
import pytest

import int4_routed_expert_02_amd as moe
from gpu_util import say
from test_gpu_linear_q4 import exact, make, run
from test_gpu_linear_q4_extremes import bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.load()


@pytest.mark.parametrize("bf16_scales", [False, True], ids=["f32", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,N,K", [(1, 96, 512), (4, 5000, 384), (7, 96, 2048), (16, 5000, 1152), (30, 80, 512), (32, 4500, 1024),
                                   (64, 48, 512), (70, 33, 384)])
@pytest.mark.parametrize("what", ["dense", "sparse", "mean 10", "sparse, mean 10"])
def test_bound(what, T, N, K, group, bf16_scales):
    import torch
    x, q, s = make(T, N, K, group, bf16_scales, seed=6)
    if "mean" in what:
        x = (x.float() + 10).to(torch.bfloat16)
    if "sparse" in what:                          # one code of 64
        g = torch.Generator(device="cuda")
        g.manual_seed(7)
        q = torch.where(torch.rand(q.shape, generator=g, device="cuda") < 1 / 32, q & 15, torch.zeros_like(q))
    ref, mag = exact(x, q, s, group)
    out = run(x, q, s).double().cpu().numpy()
    tol = bound(x, s, group, ref, mag)
    err = np.abs(out - ref) / tol
    say(f"linear {what} T={T} N={N} K={K} g={group}: {err.max():.4f} of the bound")
    assert (err <= 1).all()
