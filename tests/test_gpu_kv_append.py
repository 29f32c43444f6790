"""moe_kv_append and moe_kv_read against the formulas: norm and rotation in 64 bits, the 8-bit codes exactly from the
bf16 values, and the same bits however the rows were cut into appends.

Tolerances: norm and rotation run in f32 (mean of 64 or 128 squares, a square root's reciprocal, two products and a sum:
below 32 * 2^-24 of |a| + |b|) and round once to bf16 (8 significant bits), 2^-8 relative."""
import numpy as np
import pytest

import int4_routed_expert_02_amd as moe
from gpu_util import say
from kv_testutil import Batch, bf16_np, poison

pytestmark = pytest.mark.gpu

F32_TOL, BF16_TOL = 32 * 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.load()


def tables(n_pos, rot):
    import torch
    half = max(rot // 2, 1)
    ang = np.arange(n_pos)[:, None] * 10000.0 ** (-np.arange(half) / half)
    return (torch.from_numpy(np.cos(ang).astype(np.float32)).cuda(), torch.from_numpy(np.sin(ang).astype(np.float32)).cuda())


def rotary64(x, pos, cos, sin, rot, pairs, norm, eps):
    """[rows][heads][D] in 64 bits: (result, |a| + |b| of each value's terms)."""
    x = np.array(x, np.float64)
    if norm is not None:
        x = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * norm
    y, mag = x.copy(), np.abs(x)
    half = rot // 2
    for j in range(half):
        a, b = (2 * j, 2 * j + 1) if pairs else (j, j + half)
        c, s = cos[pos, j].astype(np.float64)[:, None], sin[pos, j].astype(np.float64)[:, None]
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
        mag[..., a] = mag[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, mag


def new_rows(b, seed=2, pad=0):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    f = torch.randn(b.rows, (b.Hq + 2 * b.H) * b.D + pad, generator=g, device="cuda").to(torch.bfloat16)
    cut = np.cumsum([0, b.Hq * b.D, b.H * b.D, b.H * b.D])
    return [f[:, cut[i]:cut[i + 1]].unflatten(1, (h, b.D)) for i, h in enumerate((b.Hq, b.H, b.H))]


def append(b, k, v, rot=None, q=None, sh=None):
    import torch
    q_out = torch.full((b.rows, b.Hq, b.D), 9.0, dtype=torch.bfloat16, device="cuda") if q is not None else None
    moe.moe_kv_append(sh if sh is not None else b.sh, b.batch, b.cache.handle, k, v, rot, q, q_out)
    torch.cuda.synchronize()
    return q_out


def codes64(vals):
    """Codes and scales of [rows][H][D] bf16 values (a whole page), by the f32 rule."""
    amax = np.abs(vals).max(axis=(0, 2)).astype(np.float32)
    scale = (amax / np.float32(127)).astype(np.float32)
    by = np.where(scale > 0, scale, np.float32(1))
    code = np.clip(np.rint((vals.astype(np.float32) / by[None, :, None]).astype(np.float32)), -127, 127)
    return code.astype(np.int64), scale


@pytest.mark.parametrize("pairs", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("dim,rot,norm", [(64, 64, True), (64, 32, False), (128, 128, True), (128, 48, True), (128, 0, True),
                                          (64, 0, False), (128, 16, False)])
def test_rotation_and_norm(dim, rot, norm, pairs):
    """q and k against 64 bits, at shifted positions too; rows apart; q in place."""
    import torch
    flags = moe.MOE_KV_ROPE_PAIRS if pairs else 0
    b = Batch([3, 40, 1], [3, 100, 65], 6, 2, dim, bits=16, page=16, flags=flags, seed=1)
    poison(b.cache)
    q, k, v = new_rows(b, pad=8)
    cos, sin = tables(5000, rot)
    g = np.random.RandomState(4)
    wq, wk = (torch.from_numpy(g.uniform(0.5, 1.5, dim).astype(np.float32)).cuda() if norm else None for _ in range(2))
    pos = np.concatenate([np.arange(l - n, l) for n, l in zip(b.new, b.lens)])
    for shift in (None, 4000):
        at = pos if shift is None else pos + shift
        rot_args = moe.kv_rotary(cos, sin, rot, None if shift is None else torch.from_numpy(at.astype(np.int32)).cuda(),
                                 wq, wk, 1e-5)
        q_out = append(b, k, v, rot_args, q)
        k_got, v_got = b.read()
        for got, x, w in ((q_out, q, wq), (k_got, k, wk)):
            ref, mag = rotary64(bf16_np(x), at, cos.cpu().numpy(), sin.cpu().numpy(), rot, pairs,
                                None if w is None else w.double().cpu().numpy(), 1e-5)
            err = np.abs(bf16_np(got) - ref) / (np.abs(ref) * BF16_TOL + mag * F32_TOL)
            say(f"rotation D={dim} rot={rot} norm={norm} shift={shift}: {err.max():.3f} of the bound")
            assert (err <= 1).all()
        assert torch.equal(v_got, v)
        q2 = q.contiguous()
        moe.moe_kv_append(b.sh, b.batch, b.cache.handle, k, v, rot_args, q2, q2)
        assert torch.equal(q2, q_out)


def test_position_outside_the_table():
    """NaN in the rotated part, the rest as it is."""
    import torch
    b = Batch([2, 2], [2, 50], 2, 2, 64, bits=16, page=16, seed=1)
    q, k, v = new_rows(b)
    cos, sin = tables(10, 32)
    q_out = append(b, k, v, moe.kv_rotary(cos, sin, 32), q)
    k_got, _ = b.read()
    for got, x in ((q_out, q), (k_got, k)):
        assert torch.isnan(got[2:, :, :32]).all() and torch.isfinite(got[:2]).all()
        assert torch.equal(got[2:, :, 32:], x[2:, :, 32:])


CUTS = {"one by one": lambda n: [1] * n, "all at once": lambda n: [n], "odd": lambda n: _odd(n),
        "pages": lambda n: [16] * (n // 16) + ([n % 16] if n % 16 else [])}


def _odd(n):
    out, sizes, i = [], [5, 39, 1, 70, 2, 17], 0
    while sum(out) < n:
        out.append(min(sizes[i % len(sizes)], n - sum(out)))
        i += 1
    return out


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("dim,page,total", [(64, 16, 147), (128, 32, 129), (64, 64, 200), (128, 128, 300)])
def test_codes_and_cuts(dim, page, total, bits):
    """Every cut of the rows into appends leaves the same bits, and in 8 bits those are the rule's."""
    import torch
    H = 3
    whole = Batch([total, total], [total, total], H, H, dim, bits=bits, page=page, seed=3)
    q, k, v = new_rows(whole)
    cos, sin = tables(total + 8, dim)
    rot = moe.kv_rotary(cos, sin, dim)
    first = None
    for name, cut in CUTS.items():
        poison(whole.cache)
        at, keys = 0, torch.empty_like(k)
        for n in cut(total):
            b = whole.sub([n, n], [at + n, at + n])
            rows = torch.cat([torch.arange(at, at + n), torch.arange(total + at, total + at + n)]).cuda()
            keys[rows] = append(b, k[rows], v[rows], rot, k[rows])   # q_out of the keys: their bf16 values
            at += n
        c = whole.cache
        used = torch.from_numpy(whole.table[:, :total // page].reshape(-1).astype(np.int64)).cuda()
        kv = [t[used].clone() for t in (c.k, c.v, c.k_scale, c.v_scale) if t is not None]
        got = whole.read()
        if first is None:
            first = (kv, got, keys.clone())
        assert all(torch.equal(x, y) for x, y in zip(kv, first[0])), name
        assert all(torch.equal(x, y) for x, y in zip(got, first[1])) and torch.equal(keys, first[2]), name
        if bits == 8:
            for s in range(2):
                kb, vb = bf16_np(keys[s * total:(s + 1) * total]), bf16_np(v[s * total:(s + 1) * total])
                for blk in range(total // page):
                    pg, at = int(whole.table[s, blk]), slice(blk * page, (blk + 1) * page)
                    for vals, codes, scales, turn in ((kb[at], c.k, c.k_scale, (1, 0, 2)), (vb[at], c.v, c.v_scale, (2, 0, 1))):
                        ref, scale = codes64(vals)
                        assert np.array_equal(scales[pg].cpu().numpy(), scale)
                        assert np.array_equal(codes[pg].cpu().numpy().transpose(turn), ref)
                open_ = slice(total // page * page, total)
                assert np.array_equal(bf16_np(got[0][s * total:(s + 1) * total])[open_], kb[open_])
                assert np.array_equal(bf16_np(got[1][s * total:(s + 1) * total])[open_], vb[open_])


@pytest.mark.parametrize("page", [16, 64])
def test_dropping_drafted_tokens(page):
    """Up to a page of the newest tokens can be dropped: other tokens in their place give what they would have given."""
    import torch
    n = 3 * page
    b = Batch([n], [n], 2, 2, 64, bits=8, page=page, seed=5)
    _, k, v = new_rows(b)
    _, k2, v2 = new_rows(b, seed=77)
    results = []
    for drafted in (0, 5, page):
        poison(b.cache)
        keep = n - page + 3 - 5                   # not at a page's start
        append(b.sub([keep], [keep]), k[:keep], v[:keep])
        for i in range(drafted):                  # refused tokens, some of which fill the page
            append(b.sub([1], [keep + i + 1]), k2[i:i + 1], v2[i:i + 1])
        append(b.sub([n - keep], [n]), k[keep:], v[keep:])
        kk, vv = b.read()
        results.append((kk, vv))
    for kk, vv in results[1:]:
        assert torch.equal(kk, results[0][0]) and torch.equal(vv, results[0][1])


@pytest.mark.parametrize("bits", [8, 16])
def test_absent_places_are_left_alone(bits):
    """Nothing is written for an absent page or slot, for rows before position 0 or from max_len on; they read as 0."""
    import torch
    b = Batch([40, 20, 5], [40, 20, 3], 2, 2, 64, bits=bits, page=16, seed=6, absent=[(0, 1)])
    poison(b.cache)
    _, k, v = new_rows(b)
    before = [t.clone() for t in (b.cache.k, b.cache.v)]
    append(b, k, v)
    kk, vv = b.read()
    gone = list(range(16, 32)) + [60, 61]         # the absent page; sequence 2's rows at positions -2 and -1
    kept = [i for i in range(65) if i not in gone]
    assert (kk[gone] == 0).all() and (vv[gone] == 0).all()
    if bits == 16:
        assert torch.equal(kk[kept], k[kept]) and torch.equal(vv[kept], v[kept])
    else:
        assert (kk[kept].float() - k[kept].float()).abs().max() < 0.05
    owned = {int(b.table[s, i]) for s, l in enumerate(b.lens) for i in range(-(-l // 16))}
    for x, y in zip((b.cache.k, b.cache.v), before):
        for pg in range(x.shape[0]):
            if pg not in owned:
                assert torch.equal(x[pg].view(torch.int8), y[pg].view(torch.int8))
    if bits == 8:                                   # a sequence without a slot
        poison(b.cache)
        b.slots[:] = [-1, 99, 1]
        b.dev_tables()
        append(b, k, v)
        assert torch.isnan(b.cache.k_scale[[int(p) for p in b.table[0, [0, 2]]]]).all()
        kk, _ = b.read()
        assert (kk[32:40] == 0).all()


def test_special_values():
    """An all-zero page has scale 0 and codes 0; an infinity or NaN makes its page and head read as NaN, and no other."""
    import torch
    b = Batch([64], [64], 2, 2, 64, bits=8, page=16, seed=8)
    _, k, v = new_rows(b)
    k, v = k.contiguous(), v.contiguous()
    k[0:16, 0] = 0
    v[16:32, 1] = -0.0
    k[35, 1, 7] = float("inf")
    v[50, 0, 3] = float("nan")
    k[50, 0] = 1e-38                                # subnormal scale
    poison(b.cache)
    append(b, k, v)
    kk, vv = b.read()
    assert (kk[0:16, 0] == 0).all() and (vv[16:32, 1] == 0).all()
    assert (b.cache.k[int(b.table[0, 0]), 0] == 0).all() and float(b.cache.k_scale[int(b.table[0, 0]), 0]) == 0.0
    nk, nv = torch.isnan(kk), torch.isnan(vv)
    assert nk[32:48, 1].all() and int(nk.sum()) == 16 * 64
    assert nv[48:64, 0].all() and int(nv.sum()) == 16 * 64


def test_rows_of_no_sequence_and_bounds():
    """rows and max_rows bound what is touched, whatever the tables hold."""
    import torch
    b = Batch([20, 6], [20, 6], 2, 2, 64, bits=16, page=16, seed=9)
    poison(b.cache)
    q, k, v = new_rows(b)
    sh = type(b.sh).from_buffer_copy(b.sh)
    sh.max_rows = 4
    q_out = append(b, k, v, None, q, sh=sh)
    took = [0, 1, 2, 3, 20, 21, 22, 23]
    left = [i for i in range(26) if i not in took]
    assert torch.equal(q_out[took], q[took]) and (q_out[left] == 9).all()
