"""The calls on a cache's pages, the attention with sinks and beam search's selection refuse what they must on the host, before
any device work, and size their workspaces; the binding refuses tensors that do not fit."""
import os

import pytest

FAKE = 1 << 20  # an aligned address that is never dereferenced: every call below fails validation first or is a no-op


@pytest.fixture(scope="module")
def moe():
    import int4_routed_expert_02_amd as m
    if not os.path.exists(m.LIB_PATH):
        from int4_routed_expert_02_amd import _build
        _build.build()
    m.load()
    return m


def shape(moe, **kw):
    base = dict(n_seq=2, rows=8, max_rows=4, max_len=100, q_heads=8, kv_heads=2, head_dim=64, kv_bits=8, page_tokens=64,
                n_pages=10, max_pages=2, n_slots=2)
    base.update(kw)
    return moe.kv_shape(**base)


class Calls:
    """Every call with good arguments but for those given."""

    def __init__(self, moe):
        self.moe, self.L = moe, moe.load()

    def batch(self, **kw):
        a = dict(row_start=FAKE, kv_len=FAKE, pages=FAKE, slots=FAKE)
        a.update(kw)
        return self.moe.MoeKvBatch(**a)

    def cache(self, **kw):
        a = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, k_tail=FAKE, v_tail=FAKE)
        a.update(kw)
        return self.moe.MoeKvCache(**a)

    def sinks(self, sh, n=4, b=None, c=None, q=FAKE, qs=512, out=FAKE, lse=None, ws=FAKE, size=1 << 40):
        return self.L.moe_kv_attention_sinks(sh, n, b or self.batch(), c or self.cache(), q, qs, out, lse, ws, size, None)

    def release(self, sh, sinks=0, kv_len=FAKE, pages=FAKE, refs=FAKE):
        return self.L.moe_kv_release(sh, sinks, kv_len, pages, refs, None)

    def fork(self, sh, b=None, parent=FAKE, kv_len=2 * FAKE, pages=2 * FAKE, slots=2 * FAKE, refs=FAKE, src=FAKE, dst=FAKE):
        return self.L.moe_kv_fork(sh, b or self.batch(), parent, kv_len, pages, slots, refs, src, dst, None)

    def reserve(self, sh, b=None, pages=FAKE, refs=FAKE, src=FAKE, dst=FAKE, missing=FAKE, ws=FAKE, size=1 << 40):
        return self.L.moe_kv_reserve(sh, b or self.batch(), pages, refs, src, dst, missing, ws, size, None)

    def compact(self, sh, pages=FAKE, refs=FAKE, moves=5, src=FAKE, dst=FAKE, live=FAKE, ws=FAKE, size=1 << 40):
        return self.L.moe_kv_compact(sh, pages, refs, moves, src, dst, live, ws, size, None)

    def copy(self, sh, c=None, n=3, src=FAKE, dst=FAKE, m=2, ssrc=FAKE, sdst=FAKE):
        return self.L.moe_kv_copy(sh, c or self.cache(), n, src, dst, m, ssrc, sdst, None)


@pytest.fixture(scope="module")
def calls(moe):
    return Calls(moe)


SHAPES = [(dict(n_seq=-1), -2), (dict(q_heads=7), -2), (dict(head_dim=96), -3), (dict(kv_bits=4), -2), (dict(page_tokens=48), -3),
          (dict(n_pages=-1), -2), (dict(max_pages=1 << 25), -2), (dict(n_slots=-1), -2), (dict(window=-1), -2)]


@pytest.mark.parametrize("kw,code", SHAPES, ids=[",".join(f"{k}={v}" for k, v in kw.items()) for kw, _ in SHAPES])
def test_shapes(moe, calls, kw, code):
    sh = shape(moe, **kw)
    for call in (calls.sinks, calls.release, calls.fork, calls.reserve, calls.compact, calls.copy):
        assert call(sh) == code
    assert moe.moe_kv_pool_workspace_bytes(sh) == 0 and moe.moe_kv_attention_sinks_workspace_bytes(sh, 4) == 0
    assert calls.release(None) == calls.copy(None) == moe.MOE_ERR_NULL


def test_null_and_alignment(moe, calls):
    sh, NULL, ALIGN = shape(moe), moe.MOE_ERR_NULL, moe.MOE_ERR_ALIGN
    for call, tables in ((calls.release, ("kv_len", "pages", "refs")), (calls.fork, ("parent", "kv_len", "pages", "slots", "refs", "src", "dst")),
                         (calls.reserve, ("pages", "refs")), (calls.compact, ("pages", "refs", "src", "dst")),
                         (calls.copy, ("src", "dst", "ssrc", "sdst"))):
        for name in tables:
            assert call(sh, **{name: None}) == NULL, name
            assert call(sh, **{name: FAKE + 2}) == ALIGN, name
    assert calls.reserve(sh, missing=FAKE + 1) == calls.compact(sh, live=FAKE + 1) == ALIGN
    wide = shape(moe, kv_bits=16)
    for name in ("src", "dst"):
        assert calls.reserve(wide, **{name: None}) == NULL and calls.reserve(wide, **{name: FAKE + 2}) == ALIGN
    for field in ("kv_len", "pages"):
        assert calls.fork(sh, b=calls.batch(**{field: None})) == NULL
        assert calls.fork(sh, b=calls.batch(**{field: FAKE + 2})) == ALIGN
    assert calls.fork(sh, b=calls.batch(slots=FAKE + 2)) == ALIGN
    for field in ("row_start", "kv_len"):
        assert calls.reserve(sh, b=calls.batch(**{field: None})) == NULL
        assert calls.reserve(sh, b=calls.batch(**{field: FAKE + 2})) == ALIGN
    for field in ("k", "v", "k_scale", "v_scale", "k_tail", "v_tail"):
        assert calls.copy(sh, c=calls.cache(**{field: None})) == NULL
        assert calls.copy(sh, c=calls.cache(**{field: FAKE + 2})) == ALIGN
    assert calls.L.moe_kv_copy(sh, None, 1, FAKE, FAKE, 0, None, None, None) == NULL
    for name in ("q", "out", "ws"):
        assert calls.sinks(sh, **{name: None}) == NULL
        assert calls.sinks(sh, **{name: FAKE + 8}) == ALIGN


def test_sizes(moe, calls):
    sh = shape(moe)
    SHAPE = moe.MOE_ERR_SHAPE
    assert calls.release(sh, sinks=-1) == calls.release(sh, sinks=(1 << 30) + 1) == SHAPE
    assert calls.sinks(sh, n=-1) == calls.sinks(sh, n=(1 << 30) + 1) == SHAPE
    assert calls.compact(sh, moves=-1) == calls.compact(sh, moves=6) == SHAPE
    assert calls.copy(sh, n=-1) == calls.copy(sh, m=-1) == SHAPE
    assert calls.fork(shape(moe, n_seq=moe.MOE_KV_FORK_MAX + 1)) == moe.MOE_ERR_UNSUPPORTED
    # rows of a fork are read while others are written
    assert calls.fork(sh, kv_len=FAKE) == calls.fork(sh, pages=FAKE) == calls.fork(sh, slots=FAKE) == SHAPE


def test_workspaces(moe, calls):
    sh = shape(moe)
    need = moe.moe_kv_pool_workspace_bytes(sh)
    assert need >= 256 and need % 256 == 0
    for call in (calls.reserve, calls.compact):
        assert call(sh, size=need - 1) == moe.MOE_ERR_WORKSPACE
        assert call(sh, size=need, ws=None) == moe.MOE_ERR_NULL
        assert call(sh, size=need, ws=FAKE + 128) == moe.MOE_ERR_ALIGN
    win = shape(moe, window=50)
    need = moe.moe_kv_attention_sinks_workspace_bytes(win, 4)
    assert need >= 256 and calls.sinks(win, size=need - 1) == moe.MOE_ERR_WORKSPACE
    assert moe.moe_kv_attention_sinks_workspace_bytes(sh, 4) == moe.moe_kv_workspace_bytes(sh)      # no window: no sinks
    assert moe.moe_kv_attention_sinks_workspace_bytes(win, 0) == moe.moe_kv_workspace_bytes(win)
    assert moe.moe_kv_attention_sinks_workspace_bytes(win, -1) == 0


def test_nothing_to_do(moe, calls):
    L = calls.L
    none = shape(moe, n_seq=0, rows=0, max_rows=0)
    assert L.moe_kv_release(none, 0, None, None, None, None) == 0
    assert L.moe_kv_release(shape(moe, max_pages=0), 0, None, None, None, None) == 0
    assert L.moe_kv_fork(none, None, None, None, None, None, None, None, None, None) == 0
    assert L.moe_kv_reserve(none, None, None, None, None, None, None, None, 0, None) == 0
    assert L.moe_kv_copy(shape(moe), None, 0, None, None, 0, None, None, None) == 0
    assert L.moe_kv_copy(shape(moe, kv_bits=16), None, 0, None, None, 5, None, None, None) == 0      # no slots in 16 bits
    assert L.moe_kv_attention_sinks(none, 4, None, None, None, 0, None, None, None, 0, None) == 0


@pytest.mark.parametrize("args,code", [
    (dict(requests=-1), -2),
    (dict(beams=0), -2),
    (dict(beams=129), -3),
    (dict(vocab=0), -2),
    (dict(vocab=(1 << 30) + 1, stride=1 << 31), -2),
    (dict(n_out=0), -2),
    (dict(n_out=129), -3),
    (dict(requests=1 << 20, beams=4), -2),
    (dict(requests=1 << 10, beams=64, vocab=1 << 21, stride=1 << 21), -2),
    (dict(fmt=2), -2),
    (dict(stride=999), -2),
    (dict(done=FAKE, end=-1), -2),
    (dict(requests=0), 0),
    (dict(logits=None), -1),
    (dict(scores=None), -1),
    (dict(parent=None), -1),
    (dict(token=None), -1),
    (dict(score=None), -1),
    (dict(ws=None), -1),
    (dict(logits=FAKE + 2), -5),
    (dict(logits=FAKE + 1, fmt=1), -5),
    (dict(scores=FAKE + 2), -5),
    (dict(lse=FAKE + 2), -5),
    (dict(token=FAKE + 1), -5),
    (dict(ws=FAKE + 128), -5),
    (dict(size=0), -4),
])
def test_beam_select(moe, args, code):
    a = dict(requests=2, beams=3, vocab=1000, n_out=4, logits=FAKE, fmt=0, stride=1000, scores=FAKE, done=None, end=5, parent=FAKE,
             token=FAKE, score=FAKE, done_out=None, lse=None, ws=FAKE, size=None)
    a.update(args)
    need = moe.moe_beam_workspace_bytes(2, 3, 1000, 4)
    assert need >= 256 and need % 256 == 0
    got = moe.load().moe_beam_select(a["requests"], a["beams"], a["vocab"], a["n_out"], a["logits"], a["fmt"], a["stride"], a["scores"],
                                     a["done"], a["end"], a["parent"], a["token"], a["score"], a["done_out"], a["lse"], a["ws"],
                                     need if a["size"] is None else a["size"], None)
    assert got == code
    assert (moe.moe_beam_workspace_bytes(a["requests"], a["beams"], a["vocab"], a["n_out"]) == 0) == \
        (code != 0 and not {"requests", "beams", "vocab", "n_out"}.isdisjoint(args))


def test_binding_refuses(moe):
    """Tensors of another type or size than the shape says never reach the library (checked before their place)."""
    import torch
    i32 = dict(dtype=torch.int32)
    sh = shape(moe)
    with pytest.raises(ValueError):
        moe.moe_kv_release(sh, 0, torch.zeros(2, dtype=torch.int64), torch.zeros(4, **i32), torch.zeros(10, **i32))
    with pytest.raises(ValueError):
        moe.moe_kv_release(sh, 0, torch.zeros(3, **i32), torch.zeros(4, **i32), torch.zeros(10, **i32))
    with pytest.raises(ValueError):
        moe.moe_kv_release(sh, 0, torch.zeros(2, **i32), torch.zeros(4, **i32), torch.zeros(10, **i32))   # not on a GPU
    x, s = torch.zeros(6, 10), torch.zeros(2, 3)
    p, t, v = torch.zeros(2, 4, **i32), torch.zeros(2, 4, **i32), torch.zeros(2, 4)
    for bad in ((x, s, p, t, v), (x[:5], s, p, t, v), (x, s, p, t.long(), v), (x, s, p, t[:1], v)):
        with pytest.raises(ValueError):
            moe.moe_beam_select(*bad)
