"""The binding's refusals with tensors on the GPU that are wrong in one property each: type, number of elements, place, gaps
between elements, shape, row stride.  What is refused has not run: the outputs keep what they held."""
import pytest

import int4_routed_expert_02_amd as moe
from kv_testutil import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.load()


N, WIDTH, PAGES = 3, 4, 20


def ints(*shape):
    import torch
    return torch.full(shape, 77, dtype=torch.int32, device="cuda")


def wrong(t):
    """(what, tensor) in which one property differs from t."""
    import torch
    flat = t.flatten()
    forms = [("type", t.long()), ("type", t.float()), ("too few", flat[:-1]), ("too many", torch.cat([flat, flat[:1]])), ("place", t.cpu())]
    return forms + ([("gaps", torch.stack([flat, flat], 1)[:, 0])] if flat.numel() > 1 else [])   # (one element has none)


def refused(call, good, names, match):
    """`call(**good)` with each of the named arguments replaced by each wrong form of it."""
    import torch
    call(**good)                                                 # the right ones pass
    before = {k: t.clone() for k, t in good.items() if torch.is_tensor(t)}
    for name in names:
        for what, bad in wrong(good[name]):
            with pytest.raises(ValueError, match=match.format(name=name)):
                call(**{**good, name: bad})
            torch.cuda.synchronize()
            for k, t in before.items():
                assert torch.equal(good[k], t), (name, what, k)


TABLE = "{name} must be a contiguous int32 GPU tensor with"


def shape(bits=16, rows=0, n_slots=N):
    return moe.kv_shape(N, rows, 1 if rows else 0, 1000, 2, 2, 64, bits, 16, PAGES, WIDTH, n_slots)


def batch(starts=None, lens=None, pages=None, slots=None):
    import torch
    starts = torch.arange(N + 1, dtype=torch.int32, device="cuda") if starts is None else starts
    lens = torch.full((N,), 5, dtype=torch.int32, device="cuda") if lens is None else lens
    return moe.kv_batch(starts, lens, ints(N, WIDTH) if pages is None else pages, ints(N) if slots is None else slots)


def workspace():
    import torch
    return torch.zeros(moe.moe_kv_pool_workspace_bytes(shape()), dtype=torch.uint8, device="cuda")


def test_release():
    good = dict(kv_len=ints(N), pages=ints(N, WIDTH), refs=ints(PAGES))
    refused(lambda **a: moe.moe_kv_release(shape(), 0, **a), good, good, TABLE)


def test_fork():
    good = dict(parent=ints(N), kv_len=ints(N), pages=ints(N, WIDTH), slots=ints(N), refs=ints(PAGES), slot_src=ints(N), slot_dst=ints(N))
    refused(lambda **a: moe.moe_kv_fork(shape(8), batch(), **a), good, good, TABLE)
    for bad in (batch(lens=ints(N - 1)), batch(pages=ints(N, WIDTH + 1)), batch(pages=ints(N + 1, WIDTH)), batch(slots=ints(N - 1))):
        with pytest.raises(ValueError, match="batch's tables"):
            moe.moe_kv_fork(shape(8), bad, **good)
    with pytest.raises(moe.MoeError):                            # in 8 bits slots and lists are needed
        moe.moe_kv_fork(shape(8), batch(), **{**good, "slots": None})


def test_reserve():
    good = dict(pages=ints(N, WIDTH), refs=ints(PAGES), copy_src=ints(N), copy_dst=ints(N), missing=ints(N), ws=workspace())
    refused(lambda **a: moe.moe_kv_reserve(shape(rows=N), batch(), **a), good, [k for k in good if k != "ws"], TABLE)
    for bad in (batch(starts=ints(N)), batch(lens=ints(N - 1))):
        with pytest.raises(ValueError, match="batch's tables"):
            moe.moe_kv_reserve(shape(rows=N), bad, **good)
    for bad in (None, good["ws"][:-256]):
        with pytest.raises(moe.MoeError):
            moe.moe_kv_reserve(shape(rows=N), batch(), **{**good, "ws": bad})
    for bad, match in ((good["ws"].cpu(), "on the GPU"), (good["ws"].repeat(2)[::2], "contiguous")):
        with pytest.raises(ValueError, match=match):
            moe.moe_kv_reserve(shape(rows=N), batch(), **{**good, "ws": bad})


def test_compact():
    good = dict(pages=ints(N, WIDTH), refs=ints(PAGES), copy_src=ints(10), copy_dst=ints(10), n_live=ints(1), ws=workspace())
    refused(lambda **a: moe.moe_kv_compact(shape(), **a), good, ("pages", "refs", "copy_dst", "n_live"), TABLE)
    for what, bad in wrong(good["copy_src"]):
        with pytest.raises(ValueError, match="copy_.* must be a contiguous int32 GPU tensor with"):
            moe.moe_kv_compact(shape(), **{**good, "copy_src": bad})
    with pytest.raises(moe.MoeError):                            # more moves than half of the pages
        moe.moe_kv_compact(shape(), **{**good, "copy_src": ints(11), "copy_dst": ints(11)})


def test_compact_without_moves():
    """No lists: nothing moves, the pages in use are counted."""
    import torch
    pages, refs, live = ints(N, WIDTH), ints(PAGES).zero_(), ints(1)
    pages.fill_(-1)
    pages[1, 0] = 13
    refs[13] = 1
    moe.moe_kv_compact(shape(), pages, refs, None, None, live, workspace())
    assert int(live) == 1 and int(pages[1, 0]) == 13 and int(refs[13]) == 1
    with pytest.raises(ValueError, match="come together"):
        moe.moe_kv_compact(shape(), pages, refs, None, ints(3), live, workspace())


@pytest.mark.parametrize("bits", [8, 16])
def test_copy(bits):
    import torch
    cache = moe.KvPages(PAGES, 2, 64, 16, bits, N if bits == 8 else 0)
    good = dict(page_src=ints(6), page_dst=ints(6), slot_src=ints(2), slot_dst=ints(2))
    call = lambda **a: moe.moe_kv_copy(shape(bits), cache.handle, **a)  # noqa: E731
    refused(call, good, ("page_dst", "slot_dst"), TABLE)
    for name in ("page_src", "slot_src"):
        for what, bad in wrong(good[name]):
            with pytest.raises(ValueError, match="must be a contiguous int32 GPU tensor with"):
                call(**{**good, name: bad})
    for name in good:
        with pytest.raises(ValueError, match="come together"):
            call(**{**good, name: None})
    other = moe.KvPages(PAGES + 1, 2, 64, 16, bits, N if bits == 8 else 0)
    with pytest.raises(ValueError, match="cache's tensors"):
        moe.moe_kv_copy(shape(bits), other.handle, **good)


def test_attention_sinks():
    import torch
    b = Batch([2, 1], [40, 70], 4, 2, 64, bits=16, page=16, window=20, seed=0)
    ws = torch.zeros(moe.moe_kv_attention_sinks_workspace_bytes(b.sh, 4), dtype=torch.uint8, device="cuda")
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    good = dict(q=q, out=torch.zeros_like(q), lse=torch.zeros(3, 4, device="cuda"), ws=ws)
    call = lambda **a: moe.moe_kv_attention_sinks(b.sh, 4, b.batch, b.cache.handle, **{**good, **a})  # noqa: E731
    call()
    wide = torch.zeros(3, 4, 128, dtype=torch.bfloat16, device="cuda")
    for name, bad, match in (("q", q.float(), "q must be a bfloat16 GPU tensor"), ("q", q.cpu(), "q must be a bfloat16 GPU tensor"),
                             ("q", q[:2], "q must be"), ("q", q[:, :3], "q must be"), ("q", wide[:, :, ::2], "contiguous"),
                             ("q", wide[:, :, :64], "contiguous"), ("out", q.float(), "out must be"), ("out", q[:2], "out must be"),
                             ("out", q.cpu(), "on the GPU"), ("out", wide[:, :, :64], "contiguous"), ("lse", good["lse"][:2], "lse must be"),
                             ("lse", good["lse"].double(), "lse must be"), ("lse", good["lse"].cpu(), "on the GPU"),
                             ("lse", torch.zeros(3, 8, device="cuda")[:, ::2], "contiguous"), ("ws", ws.cpu(), "on the GPU")):
        with pytest.raises(ValueError, match=match):
            call(**{name: bad})
    with pytest.raises(moe.MoeError):
        call(ws=None)
    with pytest.raises(moe.MoeError):
        moe.moe_kv_attention_sinks(b.sh, -1, b.batch, b.cache.handle, **good)


R, B, V, K = 2, 3, 40, 4


def beams():
    import torch
    dev = dict(device="cuda")
    return dict(logits=torch.randn(R * B, V, **dev), scores=torch.zeros(R, B, **dev), parent=ints(R, K), token=ints(R, K),
                score=torch.zeros(R, K, **dev), lse=torch.zeros(R, B, **dev), done=torch.zeros(R, B, dtype=torch.bool, **dev),
                done_out=torch.zeros(R, K, dtype=torch.uint8, **dev),
                ws=torch.zeros(moe.moe_beam_workspace_bytes(R, B, V, K), dtype=torch.uint8, **dev), end_token=3)


def test_beam_select():
    import torch
    good = beams()
    call = lambda **a: moe.moe_beam_select(**{**good, **a})  # noqa: E731
    call()
    torch.cuda.synchronize()
    before = {k: t.clone() for k, t in good.items() if torch.is_tensor(t)}
    x = good["logits"]
    cases = [("logits", t, "logits must be") for t in (x.half(), x.double(), x.long(), x[:5], x[None], x.flatten(), x.cpu())]
    cases += [("logits", torch.randn(R * B, 2 * V, device="cuda")[:, ::2], "contiguous"), ("logits", x.t().contiguous().t(), "contiguous")]
    for name in ("scores", "parent", "token", "score", "lse", "done", "done_out"):
        t = good[name]
        other = t.double() if t.dtype == torch.float32 else t.long()
        padded = torch.cat([t, t], 1)
        cases += [(name, other, f"{name} must be"), (name, t.cpu(), "on the GPU"), (name, padded[:, ::2], "contiguous"),
                  (name, padded[:, :t.shape[1]], "contiguous")]
        # another number of requests, one dimension more or less, for all but `scores` and `parent` another width too
        cases += [(name, t[:1], "must be"), (name, t[None], "must be"), (name, t.flatten(), "must be")]
        cases += [(name, padded, "must be"), (name, t[:, :-1], "must be")]
    cases += [("ws", good["ws"].cpu(), "on the GPU")]
    for name, bad, match in cases:
        with pytest.raises(ValueError, match=match):
            call(**{name: bad})
        torch.cuda.synchronize()
        for k, t in before.items():
            assert torch.equal(good[k], t), (name, k)
    for bad in (dict(ws=None), dict(ws=good["ws"][:-256]), dict(end_token=-1), dict(logits=x[:1].expand(R * B, V))):
        with pytest.raises(moe.MoeError):
            call(**bad)
