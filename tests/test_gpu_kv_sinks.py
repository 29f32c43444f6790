"""moe_kv_attention_sinks against the formula in 64 bits: windows and sinks that meet, overlap, end inside tiles and pages, lie
behind the length, with absent pages between; seeded batches of every kind.

The bound is that of the stated precision, as derived in tests/test_gpu_kv_precision.py, and 1e-30 (weights below 2^-118 of the
largest leave f32's range): the sinks add no operation to a score, a weight or a sum."""
import math
import random

import pytest

import int4_routed_expert_02_amd as moe
from kv_testutil import Batch, fill, stored
from test_gpu_kv_attention import queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.load()


def reference(b, q, sinks, max_len, max_rows):
    """out, sum w |v|, lse and the largest scale * sum |q k|, on the device in 64 bits; 99 where nothing is written."""
    import torch
    out = torch.full((b.rows, b.Hq, b.D), 99.0, dtype=torch.float64, device="cuda")
    lse, mag = torch.full((b.rows, b.Hq), 99.0, dtype=torch.float64, device="cuda"), torch.zeros_like(out)
    zmag, causal = torch.zeros_like(lse), not (b.flags & moe.MOE_KV_NONCAUSAL)
    for s, (n, length) in enumerate(zip(b.new, b.lens)):
        k, v, present = (torch.from_numpy(t).cuda() for t in stored(b, s))
        m, r = min(n, max_rows), int(b.row_start[s])
        j, p = torch.arange(length, device="cuda"), (length - n + torch.arange(m, device="cuda"))[:, None]
        sees = (present & (j < max_len)).expand(m, length).clone()
        if causal:
            sees &= j <= p
        if b.window:
            sees &= (j > p - b.window) | (j < sinks)
        for h in range(b.Hq if m else 0):
            rows, kv = q[r:r + m, h].double(), h // (b.Hq // b.H)
            z = torch.where(sees, rows @ k[:, kv].t() * b.scale, -math.inf)
            top = torch.logsumexp(z, 1)
            w = torch.where(sees, (z - torch.where(top > -math.inf, top, 0.0)[:, None]).exp(), 0.0)
            vv = torch.where(sees.any(0)[:, None], v[:, kv], 0.0) if m else v[:, kv]
            out[r:r + m, h], mag[r:r + m, h], lse[r:r + m, h] = w @ vv, w @ vv.abs(), top
            if length:
                zmag[r:r + m, h] = torch.where(sees, rows.abs() @ k[:, kv].abs().t(), 0.0).amax(1) * abs(b.scale)
    return out, mag, lse, zmag


def attend(b, q, sinks, f32=True):
    import torch
    sh = type(b.sh).from_buffer_copy(b.sh)
    sh.flags |= moe.MOE_OUT_F32 if f32 else 0
    out = torch.full((b.rows, b.Hq, b.D), 99.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    lse = torch.full((b.rows, b.Hq), 99.0, device="cuda")
    ws = torch.full((moe.moe_kv_attention_sinks_workspace_bytes(sh, sinks),), 255, dtype=torch.uint8, device="cuda")
    moe.moe_kv_attention_sinks(sh, sinks, b.batch, b.cache.handle, q, out, lse, ws)
    return out, lse


def check(b, q, sinks):
    import torch
    out, lse = attend(b, q, sinks)
    ref, mag, ref_lse, zmag = reference(b, q, sinks, b.sh.max_len, b.sh.max_rows)
    n = max(b.lens) + 1
    z_tol = (b.D / 8 + 8) * 2.0 ** -24 * zmag + 8 * 2.0 ** -24 * (zmag + 16)
    tol = mag * (2.0 ** -16 + 2.0 ** -22 + z_tol + (6 * n / 16 + 128) * 2.0 ** -24)[..., None]
    assert ((out.double() - ref).abs() <= tol + 1e-30).all()
    none = torch.isneginf(ref_lse)
    assert torch.equal(torch.isneginf(lse), none)
    assert ((lse.double() - ref_lse).abs() <= z_tol + 2.0 ** -22 + (n + 128) * 2.0 ** -24)[~none].all()
    return out, lse


SINKS = [1, 4, 15, 16, 17, 63, 64, 65, 128, 200, 100000]


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("window", [1, 40, 64, 130])
@pytest.mark.parametrize("heads,new", [((8, 2, 64), 1), ((8, 1, 128), 3), ((6, 2, 64), 40), ((8, 1, 128), 70)],
                         ids=["one", "few", "many", "many-wide"])
def test_borders(heads, new, window, page, bits):
    """Lengths around the tiles of 64 and the pages, so that sinks, window and open page meet in every way."""
    lens = [max(new, n) for n in (1, 2, 63, 64, 65, 127, 128, 129, 191, 193, 255, 257, 300, 385, 449, 520)]
    b = Batch([new] * len(lens), lens, *heads, bits=bits, page=page, window=window, seed=window + page + new)
    fill(b)
    q = queries(b)
    for sinks in SINKS:
        check(b, q, sinks)


@pytest.mark.parametrize("seed", range(60))
def test_batch(seed):
    rng = random.Random(1000 + seed)
    H, G, D = rng.choice([1, 2, 3]), rng.choice([1, 2, 3, 4, 5, 8, 16, 40]), rng.choice([64, 128])
    bits, page, most = rng.choice([8, 16]), rng.choice([16, 32, 64, 128]), rng.choice([6, 6, 150])
    new = [rng.choice([0, 1, rng.randint(1, 6), rng.randint(1, most)]) for _ in range(rng.randint(1, 5))] + [1]
    lens = [max(0, n + rng.choice([0, rng.randint(0, 20), rng.randint(0, 700), -rng.randint(0, 5), rng.randint(0, 3000)])) for n in new]
    absent = [(s, rng.randrange(max(1, -(-max(lens[s], 1) // page)))) for s in range(len(new)) if rng.random() < 0.4]
    window = rng.choice([1, rng.randint(1, 60), rng.randint(1, 300), 2 ** 31 - 1])
    max_len = rng.choice([max(lens), max(lens), rng.randint(0, max(lens))])
    b = Batch(new, lens, H * G, H, D, bits=bits, page=page, window=window, scale=rng.choice([0.0, 0.0, 0.3, -0.1]),
              flags=rng.choice([0, 0, moe.MOE_KV_NONCAUSAL]), seed=seed, absent=absent, max_len=max_len)
    b.sh.max_rows = rng.choice([max(new), max(new), rng.randint(1, max(new))])
    fill(b, seed=seed)
    check(b, queries(b, seed=seed), rng.choice([1, 4, rng.randint(1, 80), rng.randint(1, 400), 2 ** 30]))


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("new", [1, 4, 60])
def test_what_lies_between_is_not_read(new, bits):
    """Pages between sinks and window: absent or full of NaN, the same bits."""
    import torch
    lens, window, sinks, page = [1500, 700, 3000], 200, 37, 32
    b = Batch([new] * 3, lens, 8, 2, 128, bits=bits, page=page, window=window, seed=3)
    fill(b)
    q = queries(b)
    want = check(b, q, sinks)
    for s, length in enumerate(lens):
        for block in range(-(-length // page)):
            if block * page >= sinks and (block + 1) * page <= length - new - window + 1:
                pg = int(b.table[s, block])
                if bits == 16:
                    b.cache.k[pg] = b.cache.v[pg] = float("nan")
                else:
                    b.cache.k_scale[pg] = b.cache.v_scale[pg] = float("nan")
                b.table[s, block] = -1
    for _ in range(2):                                           # with NaN there, then without the pages
        got = attend(b, q, sinks)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        b.dev_tables()


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("new", [1, 50])
def test_limits(new, bits):
    """No sinks is the plain window; sinks past the length, and sinks without a window, are no window."""
    import torch
    lens = [900, 64, 333]
    b = Batch([new] * 3, lens, 8, 2, 64, bits=bits, page=64, window=100, seed=9)
    fill(b)
    q = queries(b)

    def plain(window):
        sh = type(b.sh).from_buffer_copy(b.sh)
        sh.window = window
        out, lse = torch.empty(b.rows, 8, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(b.rows, 8, device="cuda")
        ws = torch.empty(moe.moe_kv_workspace_bytes(sh), dtype=torch.uint8, device="cuda")
        moe.moe_kv_attention(sh, b.batch, b.cache.handle, q, out, lse, ws)
        return out, lse

    for got, want in ((attend(b, q, 0, False), plain(100)),):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    everything = plain(0)
    b.sh.window = 0
    got = attend(b, q, 4, False)
    assert torch.equal(got[0], everything[0]) and torch.equal(got[1], everything[1])
    b.sh.window = 100
    check(b, q, 1000)


def test_long():
    """One row over a long cache whose offsets pass 32 bits, sinks at its beginning and a window at its end."""
    import torch
    H, D, P, n_pages = 8, 128, 16, 140000                        # 140000 pages of 16384 values: above 2^31
    cache = moe.KvPages(n_pages, H, D, P, 8, 1)
    length, window, sinks = 2_000_000, 5000, 70
    per = -(-length // P)
    ids = torch.arange(n_pages - 1, n_pages - 1 - per, -1, dtype=torch.int32, device="cuda")[None].contiguous()
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    blocks = list(range(-(-sinks // P))) + list(range((length - window) // P, per))
    for block in blocks:
        pg = int(ids[0, block])
        cache.k[pg] = (torch.randn(H, P, D, generator=g, device="cuda") * 36).round().clamp(-127, 127)
        cache.v[pg] = (torch.randn(H, D, P, generator=g, device="cuda") * 36).round().clamp(-127, 127)
        cache.k_scale[pg] = cache.v_scale[pg] = 1 / 36
    q = torch.randn(1, 16, D, generator=g, device="cuda").to(torch.bfloat16)
    bt = moe.kv_batch(torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.tensor([length], dtype=torch.int32, device="cuda"), ids)
    sh = cache.shape(1, 1, 1, length, 16, per, window=window, flags=moe.MOE_OUT_F32)
    out, lse = torch.empty(1, 16, D, device="cuda"), torch.empty(1, 16, device="cuda")
    ws = torch.empty(moe.moe_kv_attention_sinks_workspace_bytes(sh, sinks), dtype=torch.uint8, device="cuda")
    moe.moe_kv_attention_sinks(sh, sinks, bt, cache.handle, q, out, lse, ws)
    pages = torch.tensor([int(ids[0, b]) for b in blocks], device="cuda")
    at = torch.tensor([b * P + i for b in blocks for i in range(P)], device="cuda")
    seen = (at < sinks) | ((at > length - 1 - window) & (at < length))
    k = cache.k[pages].double().permute(0, 2, 1, 3).reshape(-1, H, D)[seen] / 36
    v = cache.v[pages].double().permute(0, 3, 1, 2).reshape(-1, H, D)[seen] / 36
    z = torch.einsum("hd,jhd->hj", q[0].double(), k.repeat_interleave(2, 1)) / math.sqrt(D)
    w = (z - z.logsumexp(1, keepdim=True)).exp()
    want = torch.einsum("hj,jhd->hd", w, v.repeat_interleave(2, 1))
    mag = torch.einsum("hj,jhd->hd", w, v.abs().repeat_interleave(2, 1))
    assert ((out[0] - want).abs() <= mag * 2.0 ** -13 + 1e-6).all()
    assert ((lse[0] - z.logsumexp(1)).abs() <= 1e-4).all()


def test_captured():
    """A captured step replayed on other queries, with eager calls between."""
    import torch
    b = Batch([1] * 6, [700, 64, 1, 2000, 129, 65], 8, 2, 64, bits=8, page=64, window=100, seed=4)
    fill(b)
    q = queries(b).contiguous()
    out, lse = torch.empty(b.rows, 8, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(b.rows, 8, device="cuda")
    ws = torch.empty(moe.moe_kv_attention_sinks_workspace_bytes(b.sh, 5), dtype=torch.uint8, device="cuda")
    moe.moe_kv_attention_sinks(b.sh, 5, b.batch, b.cache.handle, q, out, lse, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_kv_attention_sinks(b.sh, 5, b.batch, b.cache.handle, q, out, lse, ws)
    for seed in range(3):
        q.copy_(queries(b, seed=seed))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        want = attend(b, q, 5, False)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
