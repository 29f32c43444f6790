"""Into how many parts moe_kv_attention_sinks cuts few rows behind a window, as its workspace tells (a part's partial results are
rows * q_heads * (head_dim + 2) floats; 256 bytes: not cut): no more than run at once, one workgroup a compute unit, and the same
for calls that read the same tiles of 64 positions."""
import os

import pytest


@pytest.fixture(scope="module")
def moe():
    import int4_routed_expert_02_amd as m
    if not os.path.exists(m.LIB_PATH):
        from int4_routed_expert_02_amd import _build
        _build.build()
    m.load()
    return m


def parts(moe, n, new, window, sinks, heads=(16, 4, 64), bits=8, max_len=1 << 20, flags=0):
    q_heads, kv_heads, dim = heads
    sh = moe.kv_shape(n, n * new, new, max_len, q_heads, kv_heads, dim, bits, 64, 1 << 16, max_len // 64, n, window, 0.0, flags)
    size, one = moe.moe_kv_attention_sinks_workspace_bytes(sh, sinks), n * new * q_heads * (dim + 2) * 4
    return 1 if size == 256 else round(size / one)


GROUPS = [((16, 4, 64), 8), ((16, 4, 64), 16), ((32, 8, 128), 8), ((32, 8, 128), 16)]


@pytest.mark.parametrize("heads,bits", GROUPS)
@pytest.mark.parametrize("new", [1, 3, 8])
def test_no_more_than_run_at_once(moe, heads, bits, new):
    for n in range(1, 65):
        for window in (64, 300, 512, 900, 964, 1024, 1088, 1536, 2048, 4096, 8192):
            for sinks in (1, 4, 64, 200):
                p = parts(moe, n, new, window, sinks, heads, bits)
                assert p == 1 or p * n * heads[1] <= 256, (n, window, sinks, p)


@pytest.mark.parametrize("heads,bits", GROUPS)
@pytest.mark.parametrize("new", [1, 8])
def test_neighbours(moe, heads, bits, new):
    """As windows grow parts do not become fewer; sinks of one tile are alike; one sequence fewer does not lead to many more
    parts."""
    for n in (1, 8, 16, 24, 31, 32, 33, 48, 64):
        by_window = [parts(moe, n, new, w, 4, heads, bits) for w in range(100, 4000, 37)]
        assert by_window == sorted(by_window), n
        for w in range(900, 1664, 64):
            assert parts(moe, n, new, w, 4, heads, bits) == parts(moe, n, new, w, 64, heads, bits), (n, w)
    for w in range(900, 1664, 64):
        for n in range(17, 64):
            few, many = parts(moe, n - 1, new, w, 4, heads, bits), parts(moe, n, new, w, 4, heads, bits)
            assert many <= few <= many + 1 + 256 // (n * heads[1]), (w, n, few, many)


def test_bounds(moe):
    """Short caches, windows beyond them, calls that see what follows, and windows of the largest size."""
    assert parts(moe, 1, 1, 100000, 4, max_len=64) == 1
    assert parts(moe, 1, 1, 2 ** 31 - 1, 2 ** 30, max_len=1 << 20) == 64     # 256 / 4, of 16384 tiles
    assert parts(moe, 1, 1, 64, 4, max_len=1 << 20, flags=moe.MOE_KV_NONCAUSAL) == 64   # what follows is seen
    assert parts(moe, 1, 1, 64, 4, max_len=1 << 20) == 1
    assert parts(moe, 300, 1, 4096, 4) == 1
