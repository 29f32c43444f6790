"""moe_linear_q4 with more columns than one dimension of a launch holds workgroups for: every column is computed."""
import pytest

import int4_routed_expert_02_amd as moe
from test_gpu_linear_q4 import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,N", [(33, (1 << 27) + 100), (1, (1 << 29) + 50)])
def test_every_column(T, N):
    import torch
    K = 32
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.rand(N, 1, generator=g, device="cuda") + 0.5).to(torch.bfloat16)
    out = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(moe.moe_linear_q4_workspace_bytes(T, N, K), dtype=torch.uint8, device="cuda")
    moe.moe_linear_q4(x, q, s, out, None, ws)
    assert not torch.isnan(out).any()
    for first in (0, N // 3, (1 << 26) - 500, N - 1000):
        part = slice(first, first + 1000)
        assert torch.equal(out[:, part], run(x, q[part].clone(), s[part].clone(), f32=False))
