"""moe_linear_q4 with infinite and with the largest finite activations and scales: the definition's value, infinity or
NaN (an infinity against a code of 0), not what the codes' offset makes of it.

Where the definition is finite the bound is that of the f32 sums.  A group's sum runs over x (c + 24) and -24 x, with at
most 31 and 24 of |x|: 2 * group / 32 product instructions, each adding its 32 products to the sum in at most 6 roundings
on a path.  The groups' sums, scaled, pass one rounding each and 16 more where they are joined, and the output one."""
import numpy as np
import pytest

import int4_routed_expert_02_amd as moe
from gpu_util import say
from test_gpu_linear_q4 import exact, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.load()


SIZES = [(1, 100, 512), (3, 5000, 256), (2, 17000, 96), (5, 80, 992), (16, 9000, 512), (20, 70, 512), (32, 5000, 1024), (48, 100, 512),
         (70, 33, 256)]


def codes(q):
    b = q.cpu().numpy().astype(np.int64)
    c = np.empty((b.shape[0], b.shape[1] * 2), np.int64)
    c[:, 0::2], c[:, 1::2] = b & 15, b >> 4
    return np.where(c > 7, c - 16, c)


def bound(x, s, group, ref, mag):
    wide = np.abs(x.double().cpu().numpy()) @ np.repeat(np.abs(s.double().cpu().numpy()), group, axis=1).T * 55
    return (wide * (12 * group / 32) + mag * (x.shape[1] / group + 16)) * 2.0 ** -24 + np.abs(ref) * 2.0 ** -23


@pytest.mark.parametrize("group,bf16_scales", [(32, False), (32, True), (64, True), (128, False)])
@pytest.mark.parametrize("T,N,K", SIZES)
def test_infinite_activations(T, N, K, group, bf16_scales):
    """One infinity in a token: that sign times the code's and the scale's, NaN at a code of 0; two of them, in one group
    or apart, add up as infinities do; the other tokens keep their bits."""
    import torch
    if K % group:
        K = K // group * group + group
    x, q, s = make(T, N, K, group, bf16_scales, seed=3)
    s = s.abs() + 0.001
    clean = run(x, q, s)
    c = codes(q)
    t = T - 1
    for at in ({5: np.inf}, {K - 1: -np.inf}, {0: np.inf, 1: np.inf}, {0: np.inf, K - 1: -np.inf}):
        y = x.clone()
        want = np.zeros(N)
        for k, v in at.items():
            y[t, k] = v
            with np.errstate(invalid="ignore"):
                want = want + v * c[:, k]
        got = run(y, q, s)
        g = got[t].double().cpu().numpy()
        assert np.array_equal(np.isnan(g), np.isnan(want)), at
        assert np.array_equal(g[~np.isnan(want)], want[~np.isnan(want)]), at
        keep = [i for i in range(T) if i != t]
        assert torch.equal(got[keep], clean[keep])
        half = run(y, q, s, f32=False)[t].double().cpu().numpy()
        assert np.array_equal(half, want, equal_nan=True)


@pytest.mark.parametrize("group,bf16_scales", [(32, True), (64, False), (128, True)])
@pytest.mark.parametrize("T,N,K", SIZES)
def test_largest_activations(T, N, K, group, bf16_scales):
    """Activations up to 3.38e38 whose products with small scales are far inside f32's range; a residual on top."""
    import torch
    if K % group:
        K = K // group * group + group
    x, q, s = make(T, N, K, group, bf16_scales, seed=4)
    s = s * 2.0 ** -20
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    huge = (torch.rand(T, K, generator=g, device="cuda") * 1.3e38 + 2e38) * (torch.randint(0, 2, (T, K), generator=g, device="cuda") * 2 - 1)
    x = torch.where(torch.rand(T, K, generator=g, device="cuda") < 0.05, huge, x.float()).to(torch.bfloat16)
    ref, mag = exact(x, q, s, group)
    assert np.abs(ref).max() < 1e38
    out = run(x, q, s)
    err = np.abs(out.double().cpu().numpy() - ref) / bound(x, s, group, ref, mag)
    say(f"linear T={T} N={N} K={K}, activations up to 3.3e38: {np.nanmax(err):.3f} of the bound")
    assert (err <= 1).all()
    r = torch.full((T, N), 1.5, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(run(x, q, s, r), out + 1.5)


def test_largest_scales():
    """Scales above 2.1e37 with small activations."""
    x, q, s = make(3, 200, 512, 64, False, std=1e-6)
    s = ((s.double() + 0.02) * 9e39).float()      # 1.3e38 to 3.2e38
    ref, mag = exact(x, q, s, 64)
    out = run(x, q, s)
    assert (np.abs(out.double().cpu().numpy() - ref) <= bound(x, s, 64, ref, mag)).all()
