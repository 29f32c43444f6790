"""moe_beam_select against its definition in 64 bits.

What is chosen (parents and tokens) has to be equal: the inputs' values are exact in 64 bits, and both sides' sums are off
by less than 2^-40 of the logits' range, while different sums here lie further apart (equal ones are equal on both sides,
since equal rows are summed alike).  Scores and log-sums are rounded once to f32: half a step, 2^-24 of themselves, plus the
sums' own error."""
import numpy as np
import pytest

import int4_routed_expert_02_amd as moe
from beam_testutil import select64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.load()


def call(logits, scores, n_out, done=None, end_token=-1, lse=True, ws=None, stream=None):
    """Outputs of one call, every one filled with garbage before."""
    import torch
    R, B = scores.shape
    out = dict(parent=torch.full((R, n_out), -77, dtype=torch.int32, device="cuda"),
               token=torch.full((R, n_out), -77, dtype=torch.int32, device="cuda"),
               score=torch.full((R, n_out), 7.0, device="cuda"), lse=torch.full((R, B), 7.0, device="cuda") if lse else None,
               done_out=torch.full((R, n_out), 7, dtype=torch.uint8, device="cuda"))
    if ws is None:
        ws = torch.full((moe.moe_beam_workspace_bytes(R, B, logits.shape[1], n_out),), 255, dtype=torch.uint8, device="cuda")
    moe.moe_beam_select(logits, scores, out["parent"], out["token"], out["score"], out["lse"], done, out["done_out"], end_token, ws, stream)
    return out


def check(logits, scores, n_out, done=None, end_token=-1, out=None):
    import torch
    out = out or call(logits, scores, n_out, done, end_token)
    torch.cuda.synchronize()
    want = select64(logits.double().cpu().numpy(), scores.cpu().numpy(), n_out, done.cpu().numpy() if done is not None else None,
                    end_token)
    parent, token, score, ended, lse = want
    assert np.array_equal(out["parent"].cpu().numpy(), parent)
    assert np.array_equal(out["token"].cpu().numpy(), token)
    assert np.array_equal(out["done_out"].cpu().numpy(), ended.astype(np.uint8))
    for got, ref in ((out["score"], score), (out["lse"], lse)):
        if got is None:
            continue
        got = got.cpu().numpy().astype(np.float64)
        with np.errstate(invalid="ignore", over="ignore"):
            # (a sum below the lowest f32, -3.40e38, rounds to -infinity)
            same = (got == ref.astype(np.float32)) | (np.isnan(got) & np.isnan(ref))
            near = np.abs(got - ref) <= 2.0 ** -24 * np.abs(ref) * 1.001 + 2.0 ** -38
        assert (same | near).all(), (got, ref)


def inputs(R, B, V, dtype="bf16", seed=0, std=2.5):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = (torch.randn(R * B, V, generator=g, device="cuda") * std).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    return x, -torch.rand(R, B, generator=g, device="cuda") * 6.0 - 20.0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,B,V,n", [
    (1, 1, 1, 1), (1, 1, 2, 5), (3, 2, 7, 4), (2, 3, 8, 8), (1, 4, 255, 128), (2, 2, 257, 9), (1, 128, 65, 128), (5, 1, 2047, 64),
    (2, 4, 2049, 16), (1, 3, 4097, 65), (2, 8, 8191, 33), (1, 2, 8193, 100), (70, 1, 300, 3), (4, 16, 12345, 31), (3, 100, 130, 1),
    (1, 4, 50257, 8), (1, 1, 131072, 128), (40, 8, 9001, 16), (2, 128, 10007, 128)])
def test_sizes(R, B, V, n, dtype):
    check(*inputs(R, B, V, dtype, seed=R * 1000 + B * 10 + V + n), n)


def test_rows_apart_and_unaligned():
    """Rows inside wider ones, begun at an odd element."""
    import torch
    for dtype in ("bf16", "f32"):
        wide, scores = inputs(2, 3, 5001, dtype, seed=5)
        for a, b in ((0, 4999), (1, 5001), (3, 2500), (7, 8)):
            check(wide[:, a:b], scores, 6)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equal_values(dtype):
    """All logits equal, few different ones, one row like another: the lower row, then the lower token."""
    import torch
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    for R, B, V, n in ((2, 3, 9000, 40), (1, 64, 5000, 128), (1, 4, 50257, 8), (3, 2, 33, 128)):
        scores = torch.full((R, B), -3.0, device="cuda")
        check(torch.zeros(R * B, V, dtype=dt, device="cuda"), scores, n)
        g = torch.Generator(device="cuda")
        g.manual_seed(R)
        x = torch.randint(0, 3, (R * B, V), generator=g, device="cuda").to(dt)
        check(x, scores, n)
        one = torch.randn(1, V, generator=g, device="cuda").to(dt)
        check(one.repeat(R * B, 1), scores, n)
        zeros = torch.zeros(R * B, V, dtype=dt, device="cuda")
        zeros[:, 1::2] = -0.0                                     # both zeros are one value
        check(zeros, scores, n)


def test_first_step():
    """One live beam of many, as after a prompt, wherever it is."""
    import torch
    for B, V, n, live in ((32, 131071, 64, 0), (32, 131071, 128, 21), (128, 9000, 128, 127), (8, 50257, 16, 3)):
        x, _ = inputs(2, B, V, "f32", seed=B + live)
        scores = torch.full((2, B), -float("inf"), device="cuda")
        scores[:, live] = 0.0
        check(x, scores, n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masked(dtype):
    """Logits of -infinity and of the type's lowest value; rows with nothing left; fewer candidates than asked for."""
    import torch
    low = torch.finfo(torch.bfloat16 if dtype == "bf16" else torch.float32).min
    for V, n in ((40, 16), (9000, 40), (20000, 128)):
        x, scores = inputs(3, 4, V, dtype, seed=V)
        x[0] = -float("inf")
        x[1, 5:] = -float("inf")
        x[2] = low
        x[3, ::2] = low
        x[4:8, 2:] = -float("inf")                               # request 1: two candidates a row
        x[8:12] = -float("inf")                                  # request 2: none
        x[5] = -float("inf")
        x[5, V // 2] = low
        check(x, scores, n)


def test_nan_and_infinity():
    """A row with a NaN of either sign or +infinity offers nothing; nor does a row whose score is not finite."""
    import torch
    for V in (100, 30000):
        x, scores = inputs(2, 8, V, "f32", seed=V)
        x[0, 3] = float("nan")
        x[1, V - 1] = float("inf")
        x[2, V // 2] = torch.tensor([-1], dtype=torch.int32).view(torch.float32).item()
        x.view(torch.int32)[3, 7] = -1                           # a NaN with its sign set
        x[4, 0] = float("inf")
        x[4, 1] = -float("inf")
        scores[1, 0], scores[1, 1], scores[1, 2] = float("nan"), float("inf"), -float("inf")
        check(x, scores, 12)
        check(x.to(torch.bfloat16), scores, 12)


def test_far_values():
    """Logits far apart and very large: no sum leaves the range of 64 bits."""
    import torch
    x, scores = inputs(2, 4, 5000, "f32", seed=9, std=1000.0)
    check(x, scores, 20)
    x = x * 3e34
    check(x, scores, 20)
    x = torch.full((4, 3000), -3.4e38, device="cuda")
    x[:, 7] = 3.4e38
    x[2, 1000] = 0.0
    check(x, scores[:1], 9)
    check(torch.randn(4, 3000, device="cuda") * 1e-30, scores[:1], 9)


def test_small_differences():
    """Scores that differ in their last bits decide between rows with the same logits."""
    import torch
    x, _ = inputs(1, 1, 7001, "f32", seed=3)
    x = x.repeat(6, 1)
    s = torch.tensor([-21.5], device="cuda")
    scores = torch.stack([torch.nextafter(s, s + 1), s, torch.nextafter(s, s - 1), s, s, torch.nextafter(s, s + 1)], dim=1)
    check(x, scores, 20)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,V,n", [(33, 31, 2), (16, 9000, 16), (4, 50257, 8)])
def test_one_token_allowed(B, V, n, dtype):
    """Rows that allow one token alone: its logit is the log-sum, so the beams keep their scores exactly and equal scores go
    by the row, also beside ended beams.  (-20 - x and back lose nothing: x has 24 bits from 2^-19 on, the sum 53 below 2^6.)"""
    import torch
    x, scores = inputs(2, B, V, dtype, seed=B + V)
    at = torch.randint(0, V, (2 * B, 1), device="cuda", generator=torch.Generator("cuda").manual_seed(V))
    x = torch.full_like(x, -float("inf")).scatter(1, at, x.gather(1, at))
    assert float(x[x > -float("inf")].abs().min()) > 1e-6 and float(x.max()) < 16
    scores[:] = -20.0
    scores[1, ::3] = -19.0
    check(x, scores, n)
    done = torch.zeros(2, B, dtype=torch.bool, device="cuda")
    done[:, 1::2] = True
    check(x, scores, n, done, 1)
    out = call(x, scores, n)
    assert set(out["score"].flatten().tolist()) <= {-20.0, -19.0, -float("inf")}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,B,V,n", [(16, 2, 9000, 100), (4, 8, 2000, 128), (16, 16, 4000, 64), (64, 1, 50257, 64), (1, 2, 50257, 128),
                                     (3, 1, 1105, 128), (2, 3, 808, 100), (5, 2, 129, 128), (300, 2, 8193, 120), (1, 4, 2176, 65)])
def test_many_of_few_pieces(R, B, V, n, dtype):
    """Many asked for where rows have few pieces, or a last one with few values; with values that are equal, and masked ones."""
    import torch
    x, scores = inputs(R, B, V, dtype, seed=V + n)
    check(x, scores, n)
    # equal values: the rows' sums of exponentials in any order are apart by less than the scores, which differ from row to row
    check((x / 2).round() * 2, scores, n)
    x[torch.rand(x.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(n)) < 0.95] = -float("inf")
    check(x, scores, n)


@pytest.mark.parametrize("V,n", [(11, 6), (9000, 16), (50257, 40)])
def test_done(V, n):
    """Ended beams stand still: end_token alone, at their score, also beside live ones and where all have ended."""
    import torch
    x, scores = inputs(4, 6, V, "bf16", seed=V)
    done = torch.zeros(4, 6, dtype=torch.bool, device="cuda")
    done[0, 2] = done[1, :5] = done[2] = True
    scores[1, 3] = -float("inf")
    x[9, 4] = 30.0                                               # a live row that ends now
    check(x, scores, n, done, 4)
    check(x, scores, n, done.to(torch.uint8), 0)
    x[12:18] = float("nan")                                      # logits of ended rows are not looked at for the choice
    out = call(x, scores, n, done, 4, lse=False)
    check(torch.nan_to_num(x), scores, n, done, 4, out)


def test_without_outputs_and_empty():
    import torch
    x, scores = inputs(2, 2, 100)
    out = call(x, scores, 4)
    p, t, s = (torch.empty_like(out[k]) for k in ("parent", "token", "score"))
    ws = torch.empty(moe.moe_beam_workspace_bytes(2, 2, 100, 4), dtype=torch.uint8, device="cuda")
    moe.moe_beam_select(x, scores, p, t, s, ws=ws)
    assert torch.equal(p, out["parent"]) and torch.equal(t, out["token"]) and torch.equal(s, out["score"])
    none = torch.empty(0, 4, dtype=torch.int32, device="cuda")
    moe.moe_beam_select(x[:0], scores[:0], none, none, torch.empty(0, 4, device="cuda"), ws=ws)


def test_streams_and_graph():
    """Two calls at once on streams and workspaces of their own; a captured call replayed on new inputs."""
    import torch
    a, sa = inputs(4, 8, 20011, seed=1)
    b, sb = inputs(3, 4, 50257, "f32", seed=2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):
        oa = [call(a, sa, 16) for _ in range(4)]
    with torch.cuda.stream(s2):
        ob = [call(b, sb, 9) for _ in range(4)]
    torch.cuda.synchronize()
    for o in oa:
        check(a, sa, 16, out=o)
    for o in ob:
        check(b, sb, 9, out=o)
    x, sc = a.clone(), sa.clone()
    ws = torch.empty(moe.moe_beam_workspace_bytes(4, 8, 20011, 16), dtype=torch.uint8, device="cuda")
    out = call(x, sc, 16, ws=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_beam_select(x, sc, out["parent"], out["token"], out["score"], out["lse"], None, out["done_out"], -1, ws)
    for seed in range(3, 6):
        y, sy = inputs(4, 8, 20011, seed=seed)
        x.copy_(y)
        sc.copy_(sy)
        g.replay()
        torch.cuda.synchronize()
        check(y, sy, 16, out=out)


def test_repeated_calls_give_the_same_bits():
    import torch
    x, scores = inputs(6, 8, 30001, "f32", seed=11)
    first = call(x, scores, 24)
    for _ in range(5):
        again = call(x, scores, 24)
        for k, v in first.items():
            assert torch.equal(v.view(torch.int32) if v.dtype == torch.float32 else v, again[k].view(torch.int32) if v.dtype == torch.float32 else again[k])
