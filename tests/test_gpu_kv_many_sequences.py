"""Batches of very many sequences of which one is long: what a call does goes by the rows that there are, and no valid batch
is refused for the product of its sequences and the longest one's rows.

The joint call is compared with calls on its two halves: bit for bit where the arithmetic is the same (append, read), for
attention within the two sides' own bounds (weights to 2^-16, f32 sums over at most 12000 positions, both relative to the
largest |value|)."""
import numpy as np
import pytest

import int4_routed_expert_02_amd as moe
from kv_testutil import Batch, fill, poison
from test_gpu_kv_append import append, new_rows, tables
from test_gpu_kv_attention import attend, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.load()


def batch(n_seq, longest, where, q_heads=64, kv_heads=8, dim=64, page=16, bits=16, others=1, seed=41):
    rs = np.random.RandomState(seed)
    new = np.where(rs.rand(n_seq) < 0.1, 0, others)          # some sequences without a row
    lens = new + rs.randint(0, 40, n_seq)
    new[where], lens[where] = longest, longest + 7
    return Batch(new.tolist(), lens.tolist(), q_heads, kv_heads, dim, bits=bits, page=page, seed=seed)


def halves(b, where):
    """The long sequence alone, and the others: the same cache and lengths, the other's rows left out."""
    long_new, rest_new = [0] * len(b.new), list(b.new)
    long_new[where], rest_new[where] = b.new[where], 0
    first = int(b.row_start[where])
    at = np.arange(b.rows)
    is_long = (at >= first) & (at < first + b.new[where])
    return (long_new, is_long), (rest_new, ~is_long)


def one(b, where):
    """A batch of the one sequence of b, on the same cache."""
    c = object.__new__(Batch)
    c.__dict__.update(b.__dict__)
    c.new, c.lens, c.rows = [b.new[where]], [b.lens[where]], b.new[where]
    c.table, c.slots, c.row_start = b.table[where:where + 1], b.slots[where:where + 1], np.array([0, b.new[where]], np.int32)
    c.dev_tables()
    c.sh = b.cache.shape(1, c.rows, c.rows, c.lens[0], b.Hq, b.max_pages, window=b.window, flags=b.flags)
    return c


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("n_seq,longest,where", [(3000, 12000, 1234), (5, 700, 0), (40, 1000, 39), (300, 2000, 77)])
def test_append_and_read(n_seq, longest, where, bits):
    import torch
    b = batch(n_seq, longest, where, bits=bits)
    q, k, v = new_rows(b)
    cos, sin = tables(longest + 60, 64)
    rot = moe.kv_rotary(cos, sin, 64)
    poison(b.cache)
    q_out = append(b, k, v, rot, q)
    k_got, v_got = b.read()
    held = [t.clone() for t in b.cache.handle.tensors if t is not None]
    poison(b.cache)
    want_q, want_k, want_v = (torch.empty_like(t) for t in (q_out, k_got, v_got))
    for new, mask in halves(b, where):
        rows = torch.from_numpy(np.nonzero(mask)[0]).cuda()
        c = one(b, where) if new[where] else b.sub(new, b.lens)
        assert c.sh.max_rows == max(new)
        want_q[rows] = append(c, k[rows], v[rows], rot, q[rows])
        want_k[rows], want_v[rows] = c.read()
    for got, want in ((q_out, want_q), (k_got, want_k), (v_got, want_v)):       # as bits: rows before the new ones are NaN
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    for x, y in zip(held, [t for t in b.cache.handle.tensors if t is not None]):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("bits,dim", [(8, 64), (16, 64), (8, 128)])
@pytest.mark.parametrize("n_seq,longest,where", [(3000, 12000, 2999), (40, 1000, 3)])
def test_attention(n_seq, longest, where, bits, dim):
    import torch
    b = batch(n_seq, longest, where, dim=dim, bits=bits)
    fill(b)
    q = queries(b)
    out, lse = attend(b, q)
    top = 127 * 1.5 / 36 + 1                                 # above the largest |value| that fill() makes
    for new, mask in halves(b, where):
        rows = torch.from_numpy(np.nonzero(mask)[0]).cuda()
        c = one(b, where) if new[where] else b.sub(new, b.lens)
        want, want_lse = attend(c, q[rows])
        assert torch.equal(torch.isneginf(lse[rows]), torch.isneginf(want_lse))
        assert ((out[rows] - want).abs() <= 2 * top * (2.0 ** -16 + 12000 * 2.0 ** -24)).all()
        seen = ~torch.isneginf(want_lse)
        assert ((lse[rows] - want_lse)[seen].abs() <= 2e-3).all()


def test_millions_of_sequences():
    """1.1 million sequences of one token and eight heads: more workgroups than one dimension of a launch holds."""
    import torch
    n, H, D, P = 1 << 20, 8, 64, 16
    n += 12345
    cache = moe.KvPages(64, H, D, P, 16)
    for t in (cache.k, cache.v):
        t.normal_()
    ids = (torch.arange(n, device="cuda", dtype=torch.int32) % 64)[:, None].contiguous()
    starts = torch.arange(n + 1, device="cuda", dtype=torch.int32)
    lens = (torch.arange(n, device="cuda", dtype=torch.int32) // 64 % P + 1).contiguous()
    bt = moe.kv_batch(starts, lens, ids)
    sh = cache.shape(n, n, 1, P, H, 1)
    k, v = (torch.empty(n, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    moe.moe_kv_read(sh, bt, cache.handle, k, v)
    at = torch.arange(n, device="cuda")
    assert torch.equal(k, cache.k[at % 64, :, lens.long() - 1]) and torch.equal(v, cache.v[at % 64, :, :, lens.long() - 1])
    q = k
    out = torch.zeros(n, H, D, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(moe.moe_kv_workspace_bytes(sh), dtype=torch.uint8, device="cuda")
    moe.moe_kv_attention(sh, bt, cache.handle, q, out, None, ws)
    period = 64 * P                                          # sequences this far apart are the same
    whole = n // period * period
    assert (out[:whole].unflatten(0, (-1, period)) == out[:period]).all() and torch.equal(out[whole:], out[:n - whole])
    small = cache.shape(period, period, 1, P, H, 1)
    few = torch.empty(period, H, D, dtype=torch.bfloat16, device="cuda")
    moe.moe_kv_attention(small, moe.kv_batch(starts[:period + 1], lens[:period], ids[:period]), cache.handle, q[:period], few, None, ws)
    assert torch.equal(few, out[:period])
    # append: sequences that share no page, one new token each
    own = moe.KvPages(n, 1, D, P, 16)
    ids = torch.arange(n, device="cuda", dtype=torch.int32)[:, None].contiguous()
    one_head = own.shape(n, n, 1, P, 1, 1)
    moe.moe_kv_append(one_head, moe.kv_batch(starts, lens, ids), own.handle, k[:, :1], v[:, 1:2], None, q[:, 2:3],
                      out[:, :1].contiguous())
    assert torch.equal(own.k[at, 0, lens.long() - 1], k[:, 0]) and torch.equal(own.v[at, 0, :, lens.long() - 1], v[:, 1])


def test_open_pages_of_half_a_million_sequences():
    """8 bits without a slots table: sequence s has slot s, also where a call is made in several launches."""
    import torch
    n, H, D, P = (1 << 19) + 100, 8, 64, 16                  # 34 GB of open pages
    cache = moe.KvPages(4, H, D, P, 8, n)
    cache.k_tail.normal_()
    cache.v_tail.normal_()
    ids = torch.zeros(n, 1, dtype=torch.int32, device="cuda")
    starts = torch.arange(n + 1, device="cuda", dtype=torch.int32)
    lens = (torch.arange(n, device="cuda", dtype=torch.int32) % (P - 1) + 1).contiguous()
    q = torch.randn(n, H, D, device="cuda").to(torch.bfloat16)
    out = torch.zeros_like(q)
    sh = cache.shape(n, n, 1, P, H, 1)
    ws = torch.empty(moe.moe_kv_workspace_bytes(sh), dtype=torch.uint8, device="cuda")
    moe.moe_kv_attention(sh, moe.kv_batch(starts, lens, ids), cache.handle, q, out, None, ws)
    for first in (0, (1 << 19) - 100, n - 200):
        part = slice(first, first + 200)
        some = cache.shape(200, 200, 1, P, H, 1)
        want = torch.zeros(200, H, D, dtype=torch.bfloat16, device="cuda")
        slots = torch.arange(first, first + 200, dtype=torch.int32, device="cuda")
        moe.moe_kv_attention(some, moe.kv_batch(starts[:201], lens[part].contiguous(), ids[:200], slots), cache.handle,
                             q[part].contiguous(), want, None, ws)
        assert torch.equal(out[part], want)


@pytest.mark.parametrize("bits", [8, 16])
def test_append_of_a_million_sequences(bits):
    """More workgroups than one dimension of a launch holds: the folded layout of append, a row of it partly empty."""
    import torch
    n, H, D, P = (1 << 20) + 4321, 4, 64, 16
    cache = moe.KvPages(n if bits == 16 else 8, H, D, P, bits, n if bits == 8 else 0)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    ids = torch.arange(n, device="cuda", dtype=torch.int32)[:, None].contiguous()
    starts = torch.arange(n + 1, device="cuda", dtype=torch.int32)
    lens = (torch.arange(n, device="cuda", dtype=torch.int32) % (P - 1) + 1).contiguous()       # no page fills up
    slots = torch.randperm(n, generator=g, device="cuda", dtype=torch.int32)
    if bits == 8:
        ids = ids % 8                                        # not written: the rows go to the open pages
    q, k, v = torch.randn(3, n, H, D, generator=g, device="cuda").to(torch.bfloat16)
    out = torch.zeros_like(q)
    bt = moe.kv_batch(starts, lens, ids, slots if bits == 8 else None)
    moe.moe_kv_append(cache.shape(n, n, 1, P, H, 1), bt, cache.handle, k, v, None, q, out)
    assert torch.equal(out, q)
    at, row = torch.arange(n, device="cuda"), lens.long() - 1
    if bits == 8:
        assert torch.equal(cache.k_tail[slots.long(), 0, :, row], k) and torch.equal(cache.v_tail[slots.long(), 0, :, :, row], v)
    else:
        assert torch.equal(cache.k[at, :, row], k) and torch.equal(cache.v[at, :, :, row], v)
