"""The decoder-layer operators around the MoE layer, as cases to measure: the paged key/value cache's append
(position rotation and per-head norm on the way), the attention that reads the cache (8 bits with one scale per page
and head, or bf16) and the few-token product with packed int4 weights and group scales.

A case is a dict of plain values; prepare() makes its inputs from a seed, run() is one pass (plain torch in 32 bits, or
with `own` the library's calls), exact() the definition in 64 bits and work() the bytes and operations of one pass.

Cache layout (one layer; P = tokens of a page, H = key/value heads, D = head width):
  k [pages][H][P][D], v [pages][H][D][P]: int8 codes with k_scale, v_scale [pages][H] f32, or bf16 values.
  8 bits: k_tail [slots][2][H][P][D], v_tail [slots][2][H][D][P] bf16, the rows of each sequence's two newest pages, page i
  in half i % 2; a page that is not full yet is read from there.
"""
import math
import random

import numpy as np
import torch

own = False

LARGEST = "attend_step_long"   # most bytes
WIDEST = "attend_chunk"        # most operations


def _append(name, **kw):
    return dict(dict(name=name, op="append", bits=8, page=64, rot=64, pairs=False, norm=True, shifted=False), **kw)


def _attend(name, **kw):
    return dict(dict(name=name, op="attend", bits=8, page=64, window=0, causal=True, lse=False), **kw)


def _linear(name, **kw):
    return dict(dict(name=name, op="linear", scales="f32", residual=False), **kw)


def listed():
    return [
        # one decode step of 32 sequences of the Nano model (16 query heads, 4 key/value heads of 64, per-head norm): latency
        _append("append_step", seqs=32, new=1, len=4096, q_heads=16, kv_heads=4, dim=64),
        # the prompt of a full Nano context, from an empty cache
        _append("append_prompt", seqs=1, new=4096, len=4096, q_heads=16, kv_heads=4, dim=64),
        # prompt chunks of several requests at odd places of a bf16 cache of small pages, part of each head rotated in
        # adjacent pairs, at positions of their own
        _append("append_chunks", seqs=6, new=1501, len=6007, q_heads=64, kv_heads=8, dim=128, bits=16, page=16, rot=64,
                pairs=True, norm=False, shifted=True),
        # one token of one short conversation: the smallest call
        _attend("attend_one", seqs=1, new=1, len=777, q_heads=16, kv_heads=4, dim=64),
        # the decode step that goes with append_step
        _attend("attend_step", seqs=32, new=1, len=4096, q_heads=16, kv_heads=4, dim=64),
        # decode over long documents, grouped heads, small pages
        _attend("attend_step_long", seqs=8, new=1, len=131072, q_heads=64, kv_heads=8, dim=128, page=16),
        # checking five drafted tokens of each sequence in a bf16 cache with a sliding window
        _attend("attend_verify", seqs=16, new=5, len=16384, q_heads=32, kv_heads=8, dim=128, bits=16, page=32,
                window=8192, lse=True),
        # the prompt that goes with append_prompt
        _attend("attend_prompt", seqs=1, new=4096, len=4096, q_heads=16, kv_heads=4, dim=64),
        # two prompt chunks that read a long cached beginning
        _attend("attend_chunk", seqs=2, new=2048, len=16384, q_heads=32, kv_heads=8, dim=128, page=32),
        # a Nano layer's fused q/k/v projection for one token
        _linear("linear_one", rows=1, n=1536, k=1024, group=32),
        # a wide layer's projection for the decode batch, scales in bf16, the residual added
        _linear("linear_step", rows=32, n=6144, k=8192, group=128, scales="bf16", residual=True),
        # an output head of odd width for a few tokens
        _linear("linear_odd", rows=5, n=50257, k=2048, group=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    by_name = {c["name"]: c for c in listed()}
    most_bytes, most_flops = work(by_name[LARGEST])["bytes"], work(by_name[WIDEST])["flops"]
    heads = [(16, 4, 64), (32, 8, 128), (64, 8, 128), (8, 8, 64), (12, 2, 128), (16, 1, 128), (9, 3, 64)]

    def one():
        kind = rng.choice(("append", "attend", "attend", "linear"))
        q_heads, kv_heads, dim = rng.choice(heads)
        page, bits = rng.choice((16, 32, 64, 128)), rng.choice((8, 8, 16))
        if kind == "append":
            rot = rng.choice((dim, dim, dim // 2, 0))
            new = 1 if rng.random() < 0.4 else _log(rng, 2, 8192)
            return _append(None, seqs=_log(rng, 1, 64), new=new, len=new + _log(rng, 1, 8192), q_heads=q_heads,
                           kv_heads=kv_heads, dim=dim, bits=bits, page=page, rot=rot, pairs=rng.random() < 0.5,
                           norm=rng.random() < 0.5, shifted=rng.random() < 0.3)
        if kind == "attend":
            shape = rng.random()
            new = 1 if shape < 0.4 else _log(rng, 2, 16) if shape < 0.6 else _log(rng, 17, 4096)
            length = max(_log(rng, 1, 131072 if new < 17 else 16384), new)
            return _attend(None, seqs=_log(rng, 1, 64), new=new, len=length, q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                           bits=bits, page=page, window=rng.choice((0, 0, 0, max(1, length // 3))),
                           causal=rng.random() < 0.85, lse=rng.random() < 0.5)
        group = rng.choice((32, 64, 128))
        return _linear(None, rows=_log(rng, 1, 64), n=_log(rng, 16, 50257), k=group * _log(rng, 256 // group, 12288 // group),
                       group=group, scales=rng.choice(("f32", "bf16")), residual=rng.random() < 0.5)

    got = None
    while got is None:
        c = one()
        del c["name"]
        w = work(c)
        rows, pairs = c.get("seqs", 1) * c.get("new", 1), c.get("seqs", 1) * c.get("new", 1) * c.get("len", 1) * c.get("q_heads", 1)
        if w["bytes"] <= most_bytes and w["flops"] <= most_flops and rows <= 65536 and pairs <= 1 << 31:
            got = c
    return got


# ---------------------------------------------------------------- the batch: lengths, rows, pages


def _lens(c):
    """(new rows, length after them) of each sequence: the first has the case's own, the others fewer, odd ones among them.
    In 8 bits a chunk longer than a page starts on a page, so that a pass can be repeated on the same cache."""
    i = np.arange(c["seqs"], dtype=np.int64)
    new = np.maximum(1, c["new"] - (i * 389) % (c["new"] // 2 + 1))
    length = np.maximum(new, c["len"] - (i * 7919) % (c["len"] // 2 + 1))
    if c["op"] == "append" and c["bits"] == 8:
        start = length - new
        length = np.where(new > c["page"], start - start % c["page"] + new, length)
    return new, length


def work(c):
    if c["op"] == "linear":
        t, n, k = c["rows"], c["n"], c["k"]
        size = n * k / 2 + n * k / c["group"] * (4 if c["scales"] == "f32" else 2) + t * k * 2 + t * n * (4 if c["residual"] else 2)
        return {"bytes": size, "flops": 2.0 * t * n * k}
    new, length = _lens(c)
    rows, row = float(new.sum()), c["kv_heads"] * c["dim"]
    per = c["bits"] / 8
    if c["op"] == "append":
        start = length - new
        first = start - start % c["page"]
        read = float((length - first).sum())  # rows of the touched pages, returned as the values they hold
        older = float(np.where(length // c["page"] > start // c["page"], start - first, 0).sum()) if c["bits"] == 8 else 0.0
        size = rows * (c["q_heads"] * c["dim"] * 4 + 2 * row * 2) + 2 * row * (rows * per + older * 2) + 2 * row * read * (per + 2)
        return {"bytes": size, "flops": rows * (c["q_heads"] + c["kv_heads"]) * c["dim"] * 8}
    w = c["window"] or 1 << 62
    last = np.minimum(length, w + (new - 1 if c["causal"] else 0))
    # keys of each row: all up to its own position, or the whole sequence
    keys = 0.0
    for n, l in zip(new.tolist(), length.tolist()):
        p = np.arange(l - n, l)
        keys += float((np.minimum(p + 1, w) if c["causal"] else l - np.maximum(0, p + 1 - w)).sum())
    size = 2 * row * float(last.sum()) * per + rows * c["q_heads"] * c["dim"] * 4
    return {"bytes": size, "flops": 4.0 * keys * c["q_heads"] * c["dim"]}


# ---------------------------------------------------------------- inputs


def _ints(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.int32).to(dev)


def _longs(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.int64).to(dev)


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        return (torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32) * std).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=gen, device=dev, dtype=torch.float32) * (hi - lo) + lo

    s = {"case": dict(case)}
    if case["op"] == "linear":
        t, n, k, g = case["rows"], case["n"], case["k"], case["group"]
        s["x"] = normal(t, k)
        lo = torch.randint(-7, 8, (n, k // 2), generator=gen, device=dev, dtype=torch.int8)
        hi = torch.randint(-7, 8, (n, k // 2), generator=gen, device=dev, dtype=torch.int8)
        s["q"] = ((lo & 15) | (hi << 4)).view(torch.uint8)
        s["scale"] = uniform(n, k // g, lo=0.002, hi=0.006).to(torch.float32 if case["scales"] == "f32" else torch.bfloat16)
        s["residual"] = normal(t, n) if case["residual"] else None
        s["out"] = torch.empty(t, n, dtype=torch.bfloat16, device=dev)
        return s

    new, length = _lens(case)
    S, P, H, D = case["seqs"], case["page"], case["kv_heads"], case["dim"]
    rs = np.random.RandomState(int(seed) % (1 << 32))
    per_seq = -(-length // P)
    n_pages, max_pages = int(per_seq.sum()) + 3, int(per_seq.max())
    order, table, at = rs.permutation(n_pages), np.full((S, max_pages), -1, np.int64), 0
    for i in range(S):
        table[i, :per_seq[i]] = order[at:at + per_seq[i]]
        at += int(per_seq[i])
    slots = rs.permutation(S + 1)[:S]
    row_start = np.concatenate([[0], np.cumsum(new)])
    rows = int(row_start[-1])
    s.update(rows=rows, max_rows=int(new.max()), max_len=int(length.max()), n_pages=n_pages, max_pages=max_pages, n_slots=S + 1,
             row_start=_ints(row_start, dev), kv_len=_ints(length, dev), pages=_ints(table, dev), slots=_ints(slots, dev))
    if case["bits"] == 8:
        for x, shape in (("k", (n_pages, H, P, D)), ("v", (n_pages, H, D, P))):
            codes = torch.empty(shape, dtype=torch.int8, device=dev)
            flat = codes.view(-1)
            for a in range(0, flat.numel(), 1 << 28):  # in parts: the normal values are 32 bits wide
                part = flat[a:a + (1 << 28)]
                part.copy_((torch.randn(part.numel(), generator=gen, device=dev) * 36.0).round_().clamp_(-127, 127))
            s[x] = codes
            s[x + "_scale"] = uniform(n_pages, H, lo=0.018, hi=0.036)
            s[x + "_tail"] = normal(S + 1, 2, *shape[1:])
    else:
        s["k"], s["v"] = normal(n_pages, H, P, D), normal(n_pages, H, D, P)
    if case["op"] == "attend":
        s["q"] = normal(rows, case["q_heads"], D, std=1.5)
        s["out"] = torch.empty(rows, case["q_heads"], D, dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.empty(rows, case["q_heads"], dtype=torch.float32, device=dev) if case["lse"] else None
        return s

    # one projection's output: q, k and v side by side
    fused = normal(rows, (case["q_heads"] + 2 * H) * D)
    cut = case["q_heads"] * D
    s["q"] = fused[:, :cut].unflatten(1, (case["q_heads"], D))
    s["k_new"] = fused[:, cut:cut + H * D].unflatten(1, (H, D))
    s["v_new"] = fused[:, cut + H * D:].unflatten(1, (H, D))
    s["q_norm"] = uniform(D, lo=0.5, hi=1.5) if case["norm"] else None
    s["k_norm"] = uniform(D, lo=0.5, hi=1.5) if case["norm"] else None
    start = length - new
    pos = np.concatenate([np.arange(a, a + n) for a, n in zip(start.tolist(), new.tolist())])
    shift = int(rs.randint(1, 1000)) if case["shifted"] else 0
    half = case["rot"] // 2
    angle = torch.arange(int(length.max()) + 1000, device=dev, dtype=torch.float64)[:, None] * \
        torch.pow(torch.tensor(10000.0, device=dev, dtype=torch.float64), -torch.arange(half, device=dev, dtype=torch.float64) / max(1, half))
    s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    s["pos"] = _ints(pos + shift, dev) if case["shifted"] else None
    s["q_out"] = torch.empty(rows, case["q_heads"], D, dtype=torch.bfloat16, device=dev)
    # the rows of the touched pages, by sequence: what is read back
    first = start - start % P
    count = length - first
    read_start = np.concatenate([[0], np.cumsum(count)])
    n_read = int(read_start[-1])
    s.update(n_read=n_read, max_read=int(count.max()), read_start=_ints(read_start, dev))
    s["k_read"] = torch.empty(n_read, H, D, dtype=torch.bfloat16, device=dev)
    s["v_read"] = torch.empty(n_read, H, D, dtype=torch.bfloat16, device=dev)
    # the same as index lists, for the plain form: of each row of the touched pages its sequence, position and (where new) input row
    seq = np.repeat(np.arange(S), count)
    at = np.concatenate([np.arange(a, a + n) for a, n in zip(first.tolist(), count.tolist())])
    src = row_start[seq] + at - start[seq]
    touched = np.concatenate([[0], np.cumsum(-(-count // P))])     # touched pages of each sequence, one after another
    slot_page = touched[seq] + (at - first[seq]) // P
    full = (at // P + 1) * P <= length[seq]
    lead = full & (at % P == 0)
    keep = (src >= row_start[seq]) & (at // P >= (length[seq] - 1) // P - 1)   # new rows of the two newest pages
    is_new = src >= row_start[seq]
    s["plan"] = dict(
        row_pos=_longs(pos + shift, dev), page_of=_longs(slot_page, dev), in_page=_longs(at % P, dev), n_touched=int(touched[-1]),
        src=_longs(np.maximum(src, 0), dev), is_new=torch.from_numpy(is_new).to(dev), full=torch.from_numpy(full).to(dev),
        slot=_longs(slots[seq], dev), parity=_longs(at // P % 2, dev), page_id=_longs(table[seq, at // P], dev),
        full_touched=_longs(slot_page[lead], dev), full_page=_longs(table[seq, at // P][lead], dev),
        keep_row=_longs(src[keep], dev), keep_slot=_longs(slots[seq][keep], dev), keep_half=_longs(at[keep] // P % 2, dev),
        keep_in=_longs(at[keep] % P, dev), new_page=_longs(table[seq, at // P][is_new], dev), new_in=_longs((at % P)[is_new], dev))
    return s


# ---------------------------------------------------------------- one pass


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "attend": _own_attend, "linear": _own_linear}[op](state)
    return {"append": _plain_append, "attend": _plain_attend, "linear": _plain_linear}[op](state)


def _handles(state):
    """What a program keeps beside its buffers: the shape, the batch's tables and the cache as the library takes them."""
    import int4_routed_expert_02_amd as moe
    c = state["case"]
    if c["op"] == "linear":
        state["ws"] = torch.empty(moe.moe_linear_q4_workspace_bytes(c["rows"], c["n"], c["k"]), dtype=torch.uint8, device="cuda")
        state["handles"] = moe
        return moe
    cache = moe.kv_cache(state["k"], state["v"], state.get("k_scale"), state.get("v_scale"), state.get("k_tail"), state.get("v_tail"))
    flags = 0 if c.get("causal", True) else moe.MOE_KV_NONCAUSAL
    flags |= moe.MOE_KV_ROPE_PAIRS if c.get("pairs") else 0

    def shape(rows, max_rows):
        return moe.kv_shape(n_seq=c["seqs"], rows=rows, max_rows=max_rows, max_len=state["max_len"], q_heads=c["q_heads"],
                            kv_heads=c["kv_heads"], head_dim=c["dim"], kv_bits=c["bits"], page_tokens=c["page"],
                            n_pages=state["n_pages"], max_pages=state["max_pages"], n_slots=state["n_slots"],
                            window=c.get("window", 0), flags=flags)

    def batch(row_start):
        return moe.kv_batch(row_start, state["kv_len"], state["pages"], state["slots"])

    sh = shape(state["rows"], state["max_rows"])
    if c["op"] == "attend":
        ws = torch.empty(moe.moe_kv_workspace_bytes(sh), dtype=torch.uint8, device="cuda")
        state["handles"] = (moe, sh, batch(state["row_start"]), cache, ws)
    else:
        rot = moe.kv_rotary(state["cos"], state["sin"], c["rot"], state["pos"], state["q_norm"], state["k_norm"], 1e-6)
        state["handles"] = (moe, sh, batch(state["row_start"]), cache, rot, shape(state["n_read"], state["max_read"]),
                            batch(state["read_start"]))
    return state["handles"]


def _own_append(state):
    moe, sh, batch, cache, rot, read_sh, read_batch = state.get("handles") or _handles(state)
    moe.moe_kv_append(sh, batch, cache, state["k_new"], state["v_new"], rot, state["q"], state["q_out"])
    moe.moe_kv_read(read_sh, read_batch, cache, state["k_read"], state["v_read"])
    return {"q": state["q_out"], "k": state["k_read"], "v": state["v_read"]}


def _own_attend(state):
    moe, sh, batch, cache, ws = state.get("handles") or _handles(state)
    moe.moe_kv_attention(sh, batch, cache, state["q"], state["out"], state["lse"], ws)
    return {"out": state["out"], "lse": state["lse"]}


def _own_linear(state):
    moe = state.get("handles") or _handles(state)
    moe.moe_linear_q4(state["x"], state["q"], state["scale"], state["out"], state["residual"], state["ws"])
    return state["out"]


def _plain_linear(state):
    q, scale = state["q"].view(torch.int8), state["scale"].float()
    codes = torch.stack(((q << 4) >> 4, q >> 4), dim=2).flatten(1).float()
    w = (codes.unflatten(1, (scale.shape[1], -1)) * scale[:, :, None]).flatten(1)
    y = state["x"].float() @ w.t()
    if state["residual"] is not None:
        y = y + state["residual"].float()
    return y.to(torch.bfloat16)


def _rotate(x, norm, state):
    """Norm and rotation of [rows][heads][width] values in 32 bits, rounded once."""
    c, x = state["case"], x.float()
    if norm is not None:
        x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + 1e-6) * norm
    if c["rot"]:
        cos, sin = state["cos"][state["plan"]["row_pos"]][:, None, :], state["sin"][state["plan"]["row_pos"]][:, None, :]
        r, rest = x[..., :c["rot"]], x[..., c["rot"]:]
        a, b = (r[..., 0::2], r[..., 1::2]) if c["pairs"] else (r[..., :c["rot"] // 2], r[..., c["rot"] // 2:])
        u, w = a * cos - b * sin, a * sin + b * cos
        r = torch.stack((u, w), dim=-1).flatten(-2) if c["pairs"] else torch.cat((u, w), dim=-1)
        x = torch.cat((r, rest), dim=-1)
    return x.to(torch.bfloat16)


def _plain_append(state):
    c, p = state["case"], state["plan"]
    q, k, v = _rotate(state["q"], state["q_norm"], state), _rotate(state["k_new"], state["k_norm"], state), state["v_new"]
    if c["bits"] == 16:
        state["k"][p["new_page"], :, p["new_in"], :] = k
        state["v"][p["new_page"], :, :, p["new_in"]] = v
        return {"q": q, "k": state["k"][p["page_id"], :, p["in_page"], :], "v": state["v"][p["page_id"], :, :, p["in_page"]]}

    def store(new, transposed, name):
        codes, scales, tail = state[name], state[name + "_scale"], state[name + "_tail"]
        old = tail[p["slot"], p["parity"], :, :, p["in_page"]] if transposed else tail[p["slot"], p["parity"], :, p["in_page"], :]
        rows = torch.where(p["is_new"][:, None, None], new[p["src"]], old).float()             # [touched rows][H][D]
        pages = torch.zeros(p["n_touched"], c["page"], c["kv_heads"], c["dim"], device=rows.device)
        pages[p["page_of"], p["in_page"]] = rows
        scale = pages.abs().amax(dim=(1, 3)) / 127.0                                           # [touched pages][H]
        by = torch.where(scale > 0, scale, torch.ones_like(scale))
        code = (pages / by[:, None, :, None]).round().clamp(-127, 127)
        done = code[p["full_touched"]].to(torch.int8)
        codes[p["full_page"]] = done.permute(0, 2, 3, 1) if transposed else done.permute(0, 2, 1, 3)
        scales[p["full_page"]] = scale[p["full_touched"]]
        if transposed:
            tail[p["keep_slot"], p["keep_half"], :, :, p["keep_in"]] = new[p["keep_row"]]
        else:
            tail[p["keep_slot"], p["keep_half"], :, p["keep_in"], :] = new[p["keep_row"]]
        stored = (code * scale[:, None, :, None])[p["page_of"], p["in_page"]]
        return torch.where(p["full"][:, None, None], stored, rows).to(torch.bfloat16)

    return {"q": q, "k": store(k, False, "k"), "v": store(v, True, "v")}


def _plain_attend(state):
    c = state["case"]
    S, P, H, D, G = c["seqs"], c["page"], c["kv_heads"], c["dim"], c["q_heads"] // c["kv_heads"]
    length, pages = state["kv_len"].long(), state["pages"].long()
    n_pages = pages.shape[1]
    n = state["row_start"][1:].long() - state["row_start"][:-1].long()
    present = pages.clamp(min=0)
    k, v = state["k"][present].float(), state["v"][present].float()          # [S][pages][H][P][D], [S][pages][H][D][P]
    if c["bits"] == 8:
        k *= state["k_scale"][present][..., None, None]
        v *= state["v_scale"][present][..., None, None]
        is_open = (torch.arange(n_pages, device=k.device)[None] == (length // P)[:, None])[..., None, None, None]
        slot, half = state["slots"].long(), (length // P) % 2
        k = torch.where(is_open, state["k_tail"][slot, half].float()[:, None], k)
        v = torch.where(is_open, state["v_tail"][slot, half].float()[:, None], v)
    k = k.permute(0, 2, 1, 3, 4).reshape(S, H, n_pages * P, D)
    v = v.permute(0, 2, 1, 4, 3).reshape(S, H, n_pages * P, D)
    i, j = torch.arange(state["max_rows"], device=k.device), torch.arange(n_pages * P, device=k.device)
    row = (state["row_start"][:-1].long()[:, None] + i).clamp(max=state["rows"] - 1)          # [S][rows of a sequence]
    q = state["q"][row].float().unflatten(2, (H, G)).permute(0, 2, 1, 3, 4).reshape(S, H, -1, D)
    score = (q @ k.transpose(2, 3)).mul_(1.0 / math.sqrt(D))
    pos = (length - n)[:, None] + i                                                            # [S][rows]
    seen = (j < length[:, None])[:, None, :].expand(S, i.numel(), -1)
    if c["causal"]:
        seen = seen & (j <= pos[..., None])
    if c["window"]:
        seen = seen & (j > pos[..., None] - c["window"])
    score = score.unflatten(2, (-1, G)).masked_fill_(~seen[:, None, :, None, :], -math.inf).flatten(2, 3)
    top = score.amax(dim=-1, keepdim=True)
    p = score.sub_(torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    total = p.sum(dim=-1, keepdim=True)
    out = (p @ v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + total.log()).squeeze(-1)
    out = out.unflatten(2, (-1, G)).permute(0, 2, 1, 3, 4).flatten(2, 3)                       # [S][rows][q heads][D]
    lse = lse.unflatten(2, (-1, G)).permute(0, 2, 1, 3).flatten(2, 3)
    r = torch.arange(state["rows"], device=k.device)
    seq = torch.searchsorted(state["row_start"][1:].long(), r, right=True)
    at = r - state["row_start"].long()[seq]
    return {"out": out[seq, at].to(torch.bfloat16), "lse": lse[seq, at] if c["lse"] else None}


# ---------------------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        b = s["q"].to(torch.int32)
        nib = torch.empty(case["n"], case["k"], dtype=torch.int32, device=b.device)
        nib[:, 0::2], nib[:, 1::2] = b % 16, b // 16
        w = torch.where(nib > 7, nib - 16, nib).double()
        y = torch.zeros(case["rows"], case["n"], dtype=torch.float64, device=b.device)
        g = case["group"]
        for a in range(case["k"] // g):
            y += (s["x"][:, a * g:(a + 1) * g].double() @ w[:, a * g:(a + 1) * g].t()) * s["scale"][:, a].double()
        return y + s["residual"].double() if case["residual"] else y
    new, length = _lens(case)
    P, H, D = case["page"], case["kv_heads"], case["dim"]
    first_row = np.concatenate([[0], np.cumsum(new)]).tolist()
    table, slots = s["pages"].cpu().numpy(), s["slots"].cpu().numpy()

    def of_tail(i, page):
        return s["k_tail"][slots[i], page % 2].double(), s["v_tail"][slots[i], page % 2].double().transpose(1, 2)  # [H][P][D]

    if case["op"] == "attend":
        G, outs, lses = case["q_heads"] // H, [], []
        for i in range(case["seqs"]):
            n, l = int(new[i]), int(length[i])
            ids = torch.from_numpy(table[i, :-(-l // P)]).long().cuda()
            q = s["q"][first_row[i]:first_row[i + 1]].double()
            j, p = torch.arange(l, device="cuda"), torch.arange(l - n, l, device="cuda")[:, None]
            hidden = torch.zeros(n, l, dtype=torch.bool, device="cuda")
            if case["causal"]:
                hidden |= j > p
            if case["window"]:
                hidden |= j <= p - case["window"]
            out = torch.zeros(n, H, G, D, dtype=torch.float64, device="cuda")
            lse = torch.zeros(n, H, G, dtype=torch.float64, device="cuda")
            for h in range(H):
                k, v = s["k"][ids, h].double(), s["v"][ids, h].double().transpose(1, 2)
                if case["bits"] == 8:
                    k, v = k * s["k_scale"][ids, h].double()[:, None, None], v * s["v_scale"][ids, h].double()[:, None, None]
                    if l % P:
                        tk, tv = of_tail(i, l // P)
                        k[-1], v[-1] = tk[h], tv[h]
                k, v = k.reshape(-1, D)[:l], v.reshape(-1, D)[:l]
                for g in range(G):
                    z = (q[:, h * G + g] @ k.t()) / math.sqrt(D)
                    z.masked_fill_(hidden, -math.inf)
                    m = torch.logsumexp(z, dim=1)
                    out[:, h, g] = torch.where(m[:, None] > -math.inf, (z - torch.where(m > -math.inf, m, torch.zeros_like(m))[:, None]).exp_() @ v, 0.0)
                    lse[:, h, g] = m
            outs.append(out.flatten(1, 2))
            lses.append(lse.flatten(1))
        return {"out": torch.cat(outs), "lse": torch.cat(lses) if case["lse"] else None}

    shift = s["plan"]["row_pos"]

    def rotated(x, norm):
        x = x.double()
        if norm is not None:
            x = x / ((x ** 2).sum(-1, keepdim=True) / D + 1e-6).sqrt() * norm.double()
        half = case["rot"] // 2
        cos, sin = s["cos"].double()[shift][:, None], s["sin"].double()[shift][:, None]
        y = x.clone()
        for a in range(half):
            lo, hi = (2 * a, 2 * a + 1) if case["pairs"] else (a, a + half)
            y[..., lo] = x[..., lo] * cos[..., a] - x[..., hi] * sin[..., a]
            y[..., hi] = x[..., hi] * cos[..., a] + x[..., lo] * sin[..., a]
        return y

    q, k, v = rotated(s["q"], s["q_norm"]), rotated(s["k_new"], s["k_norm"]), s["v_new"].double()
    k_all, v_all = [], []
    for i in range(case["seqs"]):
        n, l = int(new[i]), int(length[i])
        start = l - n
        for page in range(start // P, -(-l // P)):
            a, b = max(start, page * P), min(l, page * P + P)
            new_rows = slice(first_row[i] + a - start, first_row[i] + b - start)
            older = a - page * P
            for got, rows, old in ((k_all, k[new_rows], 0), (v_all, v[new_rows], 1)):
                if case["bits"] == 16:
                    if older:
                        x = s["v"][table[i, page], :, :, :older].permute(2, 0, 1) if old else s["k"][table[i, page], :, :older].transpose(0, 1)
                        rows = torch.cat((x.double(), rows))
                    got.append(rows)
                    continue
                rows = rows.to(torch.bfloat16).double() if b == page * P + P else rows
                if older:
                    rows = torch.cat((of_tail(i, page)[old][:, :older].transpose(0, 1), rows))
                if b == page * P + P:
                    scale = rows.abs().amax(dim=(0, 2), keepdim=True) / 127
                    rows = (rows / scale.clamp(min=1e-300)).round() * scale
                got.append(rows)
    return {"q": q, "k": torch.cat(k_all), "v": torch.cat(v_all)}
