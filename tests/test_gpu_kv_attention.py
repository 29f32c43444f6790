"""moe_kv_attention against the formula in 64 bits, at the lengths, masks, head layouts and pages where it can go wrong.

Tolerances: every weight exp(z - m) is rounded to 16 bits once, at most 2^-8 relative (bf16 has 8 significant bits), so an
output is off by at most 2^-8 * sum w |v|.  A score is an f32 sum of D exact products: D * 2^-24 * sum |q k| in the worst
order, tiled orders stay below (D / 8 + 8) * 2^-24 * sum |q k|; that moves lse by as much and a weight by as much relative.
Exponentials, logarithm and the f32 sums of weights and values add less than 2e-4 relative to an output and 2e-5 to
lse.  A bf16 output is rounded once more, 2^-8 of itself."""
import numpy as np
import pytest

import int4_routed_expert_02_amd as moe
from gpu_util import say
from kv_testutil import Batch, attention64, fill

pytestmark = pytest.mark.gpu

W_TOL, SUM_TOL, OUT_TOL, LSE_TOL = 2.0 ** -8, 2e-4, 2.0 ** -8, 2e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.load()


def queries(b, std=1.5, seed=5, pad=0):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    q = (torch.randn(b.rows, b.Hq * b.D + pad, generator=g, device="cuda") * std).to(torch.bfloat16)
    return q[:, :b.Hq * b.D].unflatten(1, (b.Hq, b.D))


def attend(b, q, f32=True, stream=None):
    import torch
    sh = type(b.sh).from_buffer_copy(b.sh)
    sh.flags |= moe.MOE_OUT_F32 if f32 else 0
    out = torch.full((b.rows, b.Hq, b.D), 99.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    lse = torch.full((b.rows, b.Hq), 99.0, dtype=torch.float32, device="cuda")
    ws = torch.full((moe.moe_kv_workspace_bytes(sh),), 255, dtype=torch.uint8, device="cuda")
    moe.moe_kv_attention(sh, b.batch, b.cache.handle, q, out, lse, ws, stream)
    torch.cuda.synchronize()
    return out, lse


def check(b, q, tag):
    import torch
    ref, mag, ref_lse, zmag = attention64(b, q)
    z_tol = (b.D / 8 + 8) * 2.0 ** -24 * zmag
    out, lse = attend(b, q)
    out2, lse2 = attend(b, q)
    assert torch.equal(out, out2) and torch.equal(lse, lse2), "the same call gives the same bits"
    half, _ = attend(b, q, f32=False)
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    empty = np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(got_lse), empty)
    assert (got[empty] == 0).all()
    tol = mag * (W_TOL + SUM_TOL + z_tol[..., None])
    err = np.abs(got - ref) / np.maximum(tol, 1e-30)
    herr = np.abs(half.double().cpu().numpy() - ref) / np.maximum(tol + np.abs(ref) * OUT_TOL, 1e-30)
    lerr = np.abs(got_lse - np.where(empty, 0, ref_lse))[~empty] / (LSE_TOL + z_tol[~empty]) if (~empty).any() else np.zeros(1)
    say(f"attention {tag}: out {np.nanmax(err):.3f}, bf16 out {np.nanmax(herr):.3f} of the bound, lse {lerr.max():.3f}, "
        f"{int(empty.sum())} empty rows")
    assert np.isfinite(got).all() and (err <= 1).all() and (herr <= 1).all() and (lerr <= 1).all()


HEADS = [(16, 4, 64), (8, 8, 64), (9, 3, 64), (32, 8, 128), (16, 1, 128), (40, 1, 64), (2, 2, 128)]


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "-".join(map(str, h)))
def test_one_token(heads, bits):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 200, 513]
    b = Batch([1] * len(lens), lens, *heads, bits=bits, page=64, seed=3)
    fill(b)
    check(b, queries(b), f"one token {heads} {bits} bits")


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_pages(page, bits):
    lens = [page - 1, page, page + 1, 3 * page + 7, 1000]
    b = Batch([1, 3, 1, 2, 5], lens, 8, 2, 64, bits=bits, page=page, seed=4)
    fill(b)
    check(b, queries(b), f"page {page} {bits} bits")
    b = Batch([1, 3, 1, 2, 5], lens, 8, 2, 128, bits=bits, page=page, seed=4, slots=False)
    fill(b)
    check(b, queries(b, pad=24), f"page {page} {bits} bits, wide heads, strided q")


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("heads", [(16, 4, 64), (6, 1, 128), (4, 4, 64)], ids=lambda h: "-".join(map(str, h)))
@pytest.mark.parametrize("new,lens", [([5, 1, 8], [700, 5, 8]), ([33, 64, 7], [33, 300, 7]), ([131, 1], [259, 140]),
                                      ([300], [300])], ids=["few", "mixed", "chunk", "prompt"])
def test_several_tokens(new, lens, heads, bits):
    b = Batch(new, lens, *heads, bits=bits, page=32, seed=6)
    fill(b)
    check(b, queries(b), f"new {new} of {lens}, {heads} {bits} bits")


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("window", [1, 16, 100])
@pytest.mark.parametrize("new,lens", [([1, 1, 1], [400, 99, 1]), ([70, 3], [300, 150])], ids=["one", "chunk"])
def test_window(new, lens, window, bits):
    b = Batch(new, lens, 8, 2, 64, bits=bits, page=16, window=window, seed=7)
    fill(b)
    check(b, queries(b), f"window {window}, new {new}, {bits} bits")


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("new,window", [([1, 4], 0), ([70, 33], 0), ([70, 33], 50)])
def test_not_causal(new, window, bits):
    b = Batch(new, [200, 97], 8, 2, 128, bits=bits, page=32, window=window, flags=moe.MOE_KV_NONCAUSAL, seed=8)
    fill(b)
    check(b, queries(b), f"not causal, new {new}, window {window}, {bits} bits")


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("new", [[2, 1, 3, 1], [40, 20, 17, 16]], ids=["few", "chunk"])
def test_absent_pages_and_empty_rows(new, bits):
    """Pages that are gone, rows before any key, a sequence of length 0, a sequence that lost every page."""
    absent = [(0, 0), (0, 2), (0, 3)] + [(3, i) for i in range(4)]
    b = Batch(new, [90, 0, 2, 49], 4, 2, 64, bits=bits, page=16, seed=9, absent=absent)
    fill(b)
    q = queries(b)
    check(b, q, f"absent pages, {bits} bits")
    b = Batch(new, [90, 0, 2, 49], 4, 2, 64, bits=bits, page=16, seed=9, absent=absent, window=20)
    fill(b)
    check(b, q, f"absent pages and a window, {bits} bits")


@pytest.mark.parametrize("bits", [8, 16])
def test_scale_and_large_scores(bits):
    """Scores in the hundreds, negative scales, values far from one."""
    b = Batch([1, 30], [300, 200], 8, 2, 64, bits=bits, page=32, scale=0.9, seed=10)
    fill(b, k_std=3.0, v_std=1e4)
    check(b, queries(b, std=3.0), f"large scores, {bits} bits")
    b = Batch([1, 30], [300, 200], 8, 2, 64, bits=bits, page=32, scale=-0.2, seed=10)
    fill(b, v_std=1e-6)
    check(b, queries(b), f"negative scale, {bits} bits")


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("heads", [(16, 4, 64), (16, 2, 128)], ids=lambda h: "-".join(map(str, h)))
def test_long(heads, bits):
    """Long enough to be split over many workgroups."""
    b = Batch([1, 1, 2], [30001, 77, 12345], *heads, bits=bits, page=16, seed=11)
    fill(b)
    check(b, queries(b), f"long {heads} {bits} bits")
    b = Batch([20], [20000], *heads, bits=bits, page=128, seed=12)
    fill(b)
    check(b, queries(b), f"a chunk over a long cache {heads} {bits} bits")


@pytest.mark.parametrize("bits", [8, 16])
def test_max_len_leaves_out_what_lies_beyond(bits):
    """Positions from max_len on are never used, and a larger bound changes no values beyond the tolerance."""
    b = Batch([1, 5], [300, 40], 8, 2, 64, bits=bits, page=32, seed=13, max_len=100000)
    b.sh.max_len = 100000
    fill(b)
    check(b, queries(b), f"loose bound, {bits} bits")


def test_nan_page_reaches_only_rows_that_see_it():
    """8 bits: a page whose scale is NaN gives NaN to the rows that see it, and to no others."""
    import torch
    b = Batch([70], [200], 4, 2, 64, bits=8, page=16, window=40, seed=14)
    fill(b)
    q = queries(b)
    clean, _ = attend(b, q)
    b.cache.v_scale[int(b.table[0, 9]), 1] = float("nan")   # positions 144..159, head 1
    out, _ = attend(b, q)
    pos = np.arange(130, 200)
    sees = (pos >= 144) & (pos - 40 < 159)
    bad = torch.isnan(out).any(dim=2).cpu().numpy()
    assert (bad[:, 2:] == sees[:, None]).all() and not bad[:, :2].any()
    assert torch.equal(out[~torch.from_numpy(sees).cuda()], clean[~torch.from_numpy(sees).cuda()])


def test_offsets_beyond_32_bits():
    """Pages whose byte offset passes 2^32 are read where they are."""
    import torch
    H, D, P, n_pages = 8, 128, 128, 36000          # k alone is 4.7 GB of codes
    cache = moe.KvPages(n_pages, H, D, P, 8, 1)
    ids = [n_pages - 1, 3, n_pages - 2]
    for x in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        x[ids] = 0
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    for pg in ids:
        cache.k[pg] = torch.randint(-127, 128, (H, P, D), generator=g, device="cuda", dtype=torch.int8)
        cache.v[pg] = torch.randint(-127, 128, (H, D, P), generator=g, device="cuda", dtype=torch.int8)
    cache.k_scale[ids], cache.v_scale[ids] = 0.01, 0.02
    small = moe.KvPages(3, H, D, P, 8, 1)
    for i, pg in enumerate(ids):
        for x in ("k", "v", "k_scale", "v_scale"):
            getattr(small, x)[i] = getattr(cache, x)[pg]

    def run(c, pages):
        up = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
        n = 2
        sh = c.shape(1, n, n, 3 * P, 16, 3)
        q = torch.ones(n, 16, D, dtype=torch.bfloat16, device="cuda") * 0.1
        out = torch.empty(n, 16, D, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(moe.moe_kv_workspace_bytes(sh), dtype=torch.uint8, device="cuda")
        moe.moe_kv_attention(sh, moe.kv_batch(up([0, n]), up([3 * P]), up([pages])), c.handle, q, out, None, ws)
        return out

    assert torch.equal(run(cache, ids), run(small, [0, 1, 2]))


def test_other_stream_and_graph():
    """The call is ordered on the stream it is given, and replays from a graph with the tables' new values."""
    import torch
    b = Batch([1, 3], [500, 260], 16, 4, 64, bits=8, page=64, seed=15)
    fill(b)
    q = queries(b)
    want, want_lse = attend(b, q)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got, got_lse = attend(b, q, stream=st)
    assert torch.equal(got, want) and torch.equal(got_lse, want_lse)

    out = torch.empty(b.rows, b.Hq, b.D, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(moe.moe_kv_workspace_bytes(b.sh), dtype=torch.uint8, device="cuda")
    with torch.cuda.stream(st):
        moe.moe_kv_attention(b.sh, b.batch, b.cache.handle, q, out, None, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        moe.moe_kv_attention(b.sh, b.batch, b.cache.handle, q, out, None, ws)
    for scale in (1.0, 0.5, 2.0):
        q.mul_(scale)
        want, _ = attend(b, q, f32=False)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
