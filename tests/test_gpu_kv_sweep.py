"""Seeded batches of every kind for moe_kv_attention against 64 bits: ragged and empty sequences, rows before position 0,
absent pages, windows, both directions, bounds (max_len, max_rows) below what the tables hold, slots in any order.

The bound is that of the stated precision, as derived in tests/test_gpu_kv_precision.py, and 1e-30 (weights below 2^-118 of the
largest leave f32's range); rows beyond max_rows keep what was there."""
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


def reference(b, q, max_len, max_rows):
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
            sees &= j > p - b.window
        for h in range(b.Hq if m else 0):
            rows, kv = q[r:r + m, h].double(), h // (b.Hq // b.H)
            z = (rows @ k[:, kv].t() * b.scale).masked_fill(~sees, -math.inf)
            top = torch.logsumexp(z, 1)
            w = torch.where(sees, (z - torch.where(top > -math.inf, top, 0.0)[:, None]).exp(), 0.0)
            out[r:r + m, h], mag[r:r + m, h], lse[r:r + m, h] = w @ v[:, kv], w @ v[:, kv].abs(), top
            if length:
                zmag[r:r + m, h] = (rows.abs() @ k[:, kv].abs().t() * sees).amax(1) * abs(b.scale)
    return out, mag, lse, zmag


@pytest.mark.parametrize("seed", range(60))
def test_batch(seed):
    import torch
    rng = random.Random(seed)
    H, G, D = rng.choice([1, 2, 3]), rng.choice([1, 2, 3, 4, 5, 8, 16, 40]), rng.choice([64, 128])
    bits, page, most = rng.choice([8, 16]), rng.choice([16, 32, 64, 128]), rng.choice([6, 6, 150])
    new = [rng.choice([0, 1, rng.randint(1, 6), rng.randint(1, most)]) for _ in range(rng.randint(1, 5))] + [1]
    lens = [max(0, n + rng.choice([0, rng.randint(0, 20), rng.randint(0, 700), -rng.randint(0, 5), rng.randint(0, 3000)])) for n in new]
    absent = [(s, rng.randrange(max(1, -(-max(lens[s], 1) // page)))) for s in range(len(new)) if rng.random() < 0.3]
    window = rng.choice([0, 0, 1, rng.randint(1, 300), 2 ** 31 - 1])
    max_len = rng.choice([max(lens), max(lens), rng.randint(0, max(lens))])
    max_rows = rng.choice([max(new), max(new), rng.randint(1, max(new))])
    b = Batch(new, lens, H * G, H, D, bits=bits, page=page, window=window, scale=rng.choice([0.0, 0.0, 0.3, -0.1]),
              flags=rng.choice([0, 0, moe.MOE_KV_NONCAUSAL]), seed=seed, absent=absent, max_len=max_len)
    b.sh.max_rows = max_rows
    fill(b, seed=seed)
    q = queries(b, seed=seed)
    sh = type(b.sh).from_buffer_copy(b.sh)
    sh.flags |= moe.MOE_OUT_F32
    out = torch.full((b.rows, b.Hq, D), 99.0, device="cuda")
    lse = torch.full((b.rows, b.Hq), 99.0, device="cuda")
    ws = torch.full((moe.moe_kv_workspace_bytes(sh),), 255, dtype=torch.uint8, device="cuda")
    moe.moe_kv_attention(sh, b.batch, b.cache.handle, q, out, lse, ws)
    ref, mag, ref_lse, zmag = reference(b, q, max_len, max_rows)
    n = max(lens) + 1
    z_tol = (D / 8 + 8) * 2.0 ** -24 * zmag + 8 * 2.0 ** -24 * (zmag + 16)
    tol = mag * (2.0 ** -16 + 2.0 ** -22 + z_tol + (6 * n / 16 + 128) * 2.0 ** -24)[..., None]
    assert ((out.double() - ref).abs() <= tol + 1e-30).all()
    none = torch.isneginf(ref_lse)
    assert torch.equal(torch.isneginf(lse), none)
    assert ((lse.double() - ref_lse).abs() <= z_tol + 2.0 ** -22 + (n + 128) * 2.0 ** -24)[~none].all()
