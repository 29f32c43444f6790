"""The cache, attention and few-token product calls refuse what they must on the host, before any device work, and size
their workspaces."""
import ctypes
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


SHAPES = [
    (dict(), 0),
    (dict(n_seq=-1), -2),
    (dict(rows=-1), -2),
    (dict(max_rows=9), -2),
    (dict(max_rows=-1), -2),
    (dict(max_len=-1), -2),
    (dict(q_heads=0), -2),
    (dict(q_heads=7), -2),
    (dict(kv_heads=0), -2),
    (dict(head_dim=0), -2),
    (dict(head_dim=96), -3),
    (dict(kv_bits=4), -2),
    (dict(page_tokens=0), -2),
    (dict(page_tokens=48), -3),
    (dict(page_tokens=256), -3),
    (dict(n_pages=-1), -2),
    (dict(max_pages=-1), -2),
    (dict(max_pages=1 << 25), -2),
    (dict(n_slots=-1), -2),
    (dict(window=-1), -2),
    (dict(scale=float("nan")), -2),
    (dict(scale=float("inf")), -2),
    (dict(rows=1 << 30, max_rows=1, q_heads=64), -2),
]


@pytest.mark.parametrize("kw,code", SHAPES, ids=[",".join(f"{k}={v}" for k, v in kw.items()) or "good" for kw, _ in SHAPES])
def test_shapes(moe, kw, code):
    sh, L = shape(moe, **kw), moe.load()
    b, c = moe.MoeKvBatch(FAKE, FAKE, FAKE, FAKE), moe.MoeKvCache(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE)
    assert (moe.moe_kv_workspace_bytes(sh) == 0) == (code != 0)
    if code:   # a good shape would be enqueued
        assert L.moe_kv_append(sh, b, c, None, FAKE, 128, FAKE, 128, None, 0, None, None) == code
        assert L.moe_kv_attention(sh, b, c, FAKE, 512, FAKE, None, FAKE, 1 << 40, None) == code
        assert L.moe_kv_read(sh, b, c, FAKE, FAKE, None) == code


def test_kv_arguments(moe):
    L, ok = moe.load(), shape(moe)

    def tables(**kw):
        a = dict(row_start=FAKE, kv_len=FAKE, pages=FAKE, slots=FAKE)
        a.update(kw)
        return moe.MoeKvBatch(**a)

    def cache(**kw):
        a = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, k_tail=FAKE, v_tail=FAKE)
        a.update(kw)
        return moe.MoeKvCache(**a)

    need = moe.moe_kv_workspace_bytes(ok)
    assert need >= 256 and need % 256 == 0

    def append(b=None, c=None, rot=None, k=FAKE, ks=128, v=FAKE, vs=128, q=None, qs=512, qo=None, sh=ok):
        return L.moe_kv_append(sh, b or tables(), c or cache(), rot, k, ks, v, vs, q, qs, qo, None)

    def attend(b=None, c=None, q=FAKE, qs=512, out=FAKE, lse=None, ws=FAKE, n=need, sh=ok):
        return L.moe_kv_attention(sh, b or tables(), c or cache(), q, qs, out, lse, ws, n, None)

    for call in (append, attend):
        assert call(b=tables(row_start=None)) == moe.MOE_ERR_NULL
        assert call(b=tables(kv_len=None)) == moe.MOE_ERR_NULL
        assert call(b=tables(pages=None)) == moe.MOE_ERR_NULL
        assert call(b=tables(kv_len=FAKE + 2)) == moe.MOE_ERR_ALIGN
        assert call(b=tables(slots=FAKE + 1)) == moe.MOE_ERR_ALIGN
        for f in ("k", "v", "k_scale", "v_scale", "k_tail", "v_tail"):
            assert call(c=cache(**{f: None})) == moe.MOE_ERR_NULL, f
            assert call(c=cache(**{f: FAKE + 2})) == moe.MOE_ERR_ALIGN, f
    assert append(k=None) == append(v=None) == append(q=FAKE) == moe.MOE_ERR_NULL
    assert append(ks=120) == append(vs=127) == append(q=FAKE, qo=FAKE, qs=504) == moe.MOE_ERR_SHAPE
    assert append(ks=132) == append(k=FAKE + 8) == append(v=FAKE + 2) == moe.MOE_ERR_ALIGN
    assert append(q=FAKE, qo=FAKE + 8) == append(q=FAKE + 8, qo=FAKE) == moe.MOE_ERR_ALIGN
    R = moe.MoeKvRotary
    assert append(rot=R(FAKE, FAKE, 10, 66, None, None, None, 1e-6)) == moe.MOE_ERR_SHAPE
    assert append(rot=R(FAKE, FAKE, 10, 31, None, None, None, 1e-6)) == moe.MOE_ERR_SHAPE
    assert append(rot=R(FAKE, FAKE, -1, 32, None, None, None, 1e-6)) == moe.MOE_ERR_SHAPE
    assert append(rot=R(FAKE, FAKE, 10, 24, None, None, None, 1e-6)) == moe.MOE_ERR_UNSUPPORTED
    assert append(rot=R(None, FAKE, 10, 32, None, None, None, 1e-6)) == moe.MOE_ERR_NULL
    assert append(rot=R(FAKE + 4, FAKE, 10, 32, None, None, None, 1e-6)) == moe.MOE_ERR_ALIGN
    assert append(rot=R(FAKE, FAKE, 10, 32, None, FAKE + 8, None, 1e-6)) == moe.MOE_ERR_ALIGN
    assert attend(q=None) == attend(out=None) == attend(ws=None) == moe.MOE_ERR_NULL
    assert attend(qs=500) == moe.MOE_ERR_SHAPE
    assert attend(qs=516) == attend(out=FAKE + 8) == attend(lse=FAKE + 2) == attend(ws=FAKE + 16) == moe.MOE_ERR_ALIGN
    assert attend(n=need - 1) == moe.MOE_ERR_WORKSPACE
    assert L.moe_kv_read(ok, tables(), cache(), None, FAKE, None) == moe.MOE_ERR_NULL
    assert L.moe_kv_read(ok, tables(), cache(), FAKE, FAKE + 2, None) == moe.MOE_ERR_ALIGN
    for empty in (dict(rows=0, max_rows=0), dict(n_seq=0), dict(max_rows=0)):
        sh = shape(moe, **empty)
        assert L.moe_kv_append(sh, None, None, None, None, 0, None, 0, None, 0, None, None) == 0
        assert L.moe_kv_attention(sh, None, None, None, 0, None, None, None, 0, None) == 0
        assert L.moe_kv_read(sh, None, None, None, None, None) == 0
    assert L.moe_kv_append(None, None, None, None, None, 0, None, 0, None, 0, None, None) == moe.MOE_ERR_NULL


@pytest.mark.parametrize("args,code", [
    (dict(T=-1), -2),
    (dict(N=-1), -2),
    (dict(K=0), -2),
    (dict(group=0), -2),
    (dict(K=1000, stride=1000), -2),
    (dict(group=16), -3),
    (dict(group=256), -3),
    (dict(K=(1 << 26) + 32, stride=1 << 27), -3),
    (dict(stride=(1 << 25) + 8), -3),
    (dict(stride=1016), -2),
    (dict(fmt=2), -2),
    (dict(T=0), 0),
    (dict(N=0), 0),
    (dict(x=None), -1),
    (dict(q=None), -1),
    (dict(scales=None), -1),
    (dict(out=None), -1),
    (dict(ws=None), -1),
    (dict(x=FAKE + 8), -5),
    (dict(stride=1028), -5),
    (dict(q=FAKE + 8), -5),
    (dict(scales=FAKE + 8), -5),
    (dict(residual=FAKE + 1), -5),
    (dict(out=FAKE + 2, flags=1), -5),
    (dict(out=FAKE + 1), -5),
    (dict(ws=FAKE + 128), -5),
    (dict(ws_bytes=0), -4),
])
def test_linear_q4_validation(moe, args, code):
    a = dict(T=4, N=100, K=1024, group=32, x=FAKE, stride=1024, q=FAKE, scales=FAKE, fmt=0, residual=None, out=FAKE, flags=0,
             ws=FAKE, ws_bytes=None)
    a.update(args)
    need = moe.moe_linear_q4_workspace_bytes(4, 100, 1024)
    assert need >= 256
    got = moe.load().moe_linear_q4(a["T"], a["N"], a["K"], a["group"], a["x"], a["stride"], a["q"], a["scales"], a["fmt"],
                                   a["residual"], a["out"], a["flags"], a["ws"],
                                   need if a["ws_bytes"] is None else a["ws_bytes"], None)
    assert got == code
    assert moe.moe_linear_q4_workspace_bytes(-1, 4, 64) == moe.moe_linear_q4_workspace_bytes(1, 4, 0) == 0


def test_struct_sizes(moe):
    """The ctypes structs are laid out as the header's."""
    assert ctypes.sizeof(moe.MoeKvShape) == 15 * 4 and ctypes.sizeof(moe.MoeKvBatch) == 4 * 8
    assert ctypes.sizeof(moe.MoeKvCache) == 6 * 8 and ctypes.sizeof(moe.MoeKvRotary) == 56
