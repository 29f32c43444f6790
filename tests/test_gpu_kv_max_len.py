"""A max_len below a sequence's length leaves out the positions from it on and changes nothing of what lies below: a page
that is full by the sequence's length is read from its codes, wherever max_len cuts it.

The values are compared with 64 bits under the bound that tests/test_gpu_kv_attention.py derives, or bit for bit."""
import numpy as np
import pytest

import int4_routed_expert_02_amd as moe
import kv_testutil
from kv_testutil import Batch, fill, poison
from test_gpu_kv_append import append, new_rows, tables
from test_gpu_kv_attention import check, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.load()


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("window", [0, 230])
@pytest.mark.parametrize("dim,page,cut", [(64, 32, 100), (128, 16, 97), (64, 64, 130), (128, 128, 200), (64, 32, 96), (64, 16, 1)])
@pytest.mark.parametrize("new", [[1, 3, 1], [90, 40, 7]], ids=["few", "many"])
def test_attention(new, dim, page, cut, window, bits, monkeypatch):
    whole = kv_testutil.stored

    def below_cut(b, s):
        k, v, present = whole(b, s)
        return k, v, present & (np.arange(len(present)) < cut)

    b = Batch(new, [300, 205, 50], 8, 2, dim, bits=bits, page=page, window=window, seed=21, max_len=cut)
    fill(b)
    monkeypatch.setattr(kv_testutil, "stored", below_cut)
    check(b, queries(b), f"max_len {cut}, page {page}, new {new}, window {window}, {bits} bits")


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("page,cut", [(16, 97), (32, 100), (64, 130), (128, 200), (32, 96), (64, 1), (32, 0)])
def test_append_and_read(page, cut, bits):
    import torch
    lens = [300, 205, 50]
    b = Batch(lens, lens, 3, 3, 64, bits=bits, page=page, seed=22)
    _, k, v = new_rows(b)
    cos, sin = tables(400, 64)
    rot = moe.kv_rotary(cos, sin, 64)
    poison(b.cache)
    append(b, k, v, rot)
    want = b.read()
    tensors = [t for t in (b.cache.k, b.cache.v, b.cache.k_scale, b.cache.v_scale) if t is not None]
    stored = [t.clone() for t in tensors]
    pos = torch.cat([torch.arange(n) for n in lens]).cuda()

    def read_below_cut():
        b.sh.max_len = cut
        got = b.read()
        b.sh.max_len = max(lens)
        for x, y in zip(got, want):
            assert torch.equal(x, torch.where((pos < cut)[:, None, None], y, torch.zeros_like(y)))

    read_below_cut()                                       # a smaller bound when reading
    poison(b.cache)
    before = [t.clone() for t in tensors]
    b.sh.max_len = cut
    append(b, k, v, rot)                                   # and when appending
    read_below_cut()
    first_out = -(-cut // page)                            # pages from here on hold positions from max_len on only
    for s, n in enumerate(lens):
        for block in range(first_out, -(-n // page)):
            pg = int(b.table[s, block])
            for t, was in zip(tensors, before):
                assert torch.equal(t[pg].view(torch.uint8), was[pg].view(torch.uint8))
    rest = [max(n - cut, 0) for n in lens]                 # the rows that were left out, appended later
    rows = torch.cat([torch.arange(int(b.row_start[s]) + n - r, int(b.row_start[s]) + n) for s, (n, r) in enumerate(zip(lens, rest))])
    later = b.sub(rest, lens)
    append(later, k[rows.cuda()], v[rows.cuda()], rot)
    used = torch.tensor([int(b.table[s, i]) for s, n in enumerate(lens) for i in range(n // page)], dtype=torch.long).cuda()
    assert all(torch.equal(t[used], w[used]) for t, w in zip(tensors, stored))
    assert all(torch.equal(x, y) for x, y in zip(b.read(), want))
