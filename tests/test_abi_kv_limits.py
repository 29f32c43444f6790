"""Limits that the cache and product calls check on the host beside those of tests/test_abi_kv.py."""
import os

import pytest

FAKE = 1 << 20  # an aligned address that is never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def moe():
    import int4_routed_expert_02_amd as m
    if not os.path.exists(m.LIB_PATH):
        from int4_routed_expert_02_amd import _build
        _build.build()
    m.load()
    return m


def shape(moe, **kw):
    base = dict(n_seq=2, rows=8, max_rows=4, max_len=100, q_heads=8, kv_heads=2, head_dim=64, kv_bits=16, page_tokens=64,
                n_pages=10, max_pages=2, n_slots=0)
    base.update(kw)
    return moe.kv_shape(**base)


def append_in_place(moe, sh, stride):
    b, c = moe.MoeKvBatch(FAKE, FAKE, FAKE, FAKE), moe.MoeKvCache(FAKE, FAKE, None, None, None, None)
    # rot_dim's tables are missing, so a call that passes the check of q is refused all the same
    rot = moe.MoeKvRotary(None, None, 10, 32, None, None, None, 1e-6)
    return moe.load().moe_kv_append(sh, b, c, rot, FAKE, 128, FAKE, 128, FAKE, stride, FAKE, None)


def test_queries_in_place_need_their_own_places(moe):
    """Rotated in place, a row must end where it began: rows of a fused projection would be overwritten before they are read."""
    assert append_in_place(moe, shape(moe), 768) == moe.MOE_ERR_SHAPE
    assert append_in_place(moe, shape(moe), 512) == moe.MOE_ERR_NULL
    assert append_in_place(moe, shape(moe, rows=1, max_rows=1, n_seq=1), 768) == moe.MOE_ERR_NULL


@pytest.mark.parametrize("kw,good", [
    (dict(q_heads=1 << 22, kv_heads=1, n_seq=1, rows=1, max_rows=1), True),
    (dict(q_heads=(1 << 22) + 1, kv_heads=1, n_seq=1, rows=1, max_rows=1), False),
    (dict(n_seq=(1 << 26) - 1, kv_heads=1), True),
    (dict(n_seq=1 << 26, kv_heads=1), False),
    (dict(rows=(1 << 26) - 1, q_heads=1, kv_heads=1), True),
    (dict(rows=1 << 26, q_heads=1, kv_heads=1), False),
])
def test_sizes(moe, kw, good):
    assert (moe.moe_kv_workspace_bytes(shape(moe, **kw)) > 0) == good


@pytest.mark.parametrize("K,stride,code", [(1 << 25, 1 << 25, -1), ((1 << 25) + 32, (1 << 25) + 32, -3), (32, (1 << 25) + 8, -3)])
def test_longest_row_of_a_product(moe, K, stride, code):
    got = moe.load().moe_linear_q4(2, 1, K, 32, None, stride, FAKE, FAKE, 0, None, FAKE, 0, FAKE, 256, None)
    assert got == code
