"""moe_kv_attention_sinks on both sides of where few rows are cut into fewer parts: numbers of sequences, windows and rows around the
borders, against the formula in 64 bits (the bound of tests/test_gpu_kv_sinks.py)."""
import pytest

import int4_routed_expert_02_amd as moe
from kv_testutil import Batch, fill
from test_gpu_kv_attention import queries
from test_gpu_kv_sinks import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.load()


@pytest.mark.parametrize("dim,bits", [(64, 8), (64, 16), (128, 8), (128, 16)])
@pytest.mark.parametrize("n", [5, 15, 16, 17, 33])
def test_around_the_borders(n, dim, bits):
    """8 key/value heads: 256 / 8 sequences are one workgroup a compute unit, half of them two parts each."""
    for window, new in ((447, 1), (449, 3), (961, 1), (1500, 16)):
        lens = [max(new, window + 150 - 97 * (i % 7) * (i % 3)) for i in range(n)]
        b = Batch([new] * n, lens, 8, 8, dim, bits=bits, page=64, window=window, seed=n + window)
        fill(b)
        q = queries(b)
        for sinks in (4, 65):
            check(b, q, sinks)
