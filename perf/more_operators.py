"""The operators of serving over the paged cache beside its append and attention, as cases to measure: attention with a
sliding window and a few first tokens that stay visible (sinks), the cache's counted pages (forked for beams, handed out,
given back, moved together) and beam search's selection over a request's beams and the vocabulary.

A case is a dict of plain values; prepare() makes its inputs from a seed, run() is one pass (plain torch, or with `own` the
library's calls), exact() the definition in 64 bits and work() the bytes and operations of one pass.

Cache layout (one layer; P = tokens of a page, H = key/value heads, D = head width):
  k [pages][H][P][D], v [pages][H][D][P]: int8 codes with k_scale, v_scale [pages][H] f32, or bf16 values.
  8 bits: k_tail [slots][2][H][P][D], v_tail [slots][2][H][D][P] bf16, the rows of each sequence's two newest pages, page i
  in half i % 2; a page that is not full yet is read from there.
Tables: pages [sequences][blocks] i32 (-1: no page), refs [pages] i32: how many entries name the page.
"""
import math
import random

import numpy as np
import torch

own = False

LARGEST = "sinks_long"     # most bytes
WIDEST = "sinks_chunk"     # most operations


def _sinks(name, **kw):
    return dict(dict(name=name, op="sinks", bits=8, page=64, causal=True, lse=False), **kw)


def _fork(name, **kw):
    return dict(dict(name=name, op="fork", bits=8, page=64, new=1, prompt=False), **kw)


def _compact(name, **kw):
    return dict(dict(name=name, op="compact", bits=8, page=64, window=0, sinks=0, ended=3, moves=0), **kw)


def _beam(name, **kw):
    return dict(dict(name=name, op="beam", logits="bf16", done=False), **kw)


def listed():
    return [
        # a decode step of 32 conversations of the Nano model that have outgrown a window of 1024, four sinks
        _sinks("sinks_step", seqs=32, new=1, len=4096, q_heads=16, kv_heads=4, dim=64, window=1024, sinks=4),
        # decode over long documents, grouped heads, small pages, a long window and a whole instruction kept visible
        _sinks("sinks_long", seqs=8, new=1, len=131072, q_heads=64, kv_heads=8, dim=128, page=16, window=98304, sinks=500),
        # checking five drafted tokens of each sequence in a bf16 cache
        _sinks("sinks_verify", seqs=16, new=5, len=16384, q_heads=32, kv_heads=8, dim=128, bits=16, page=32, window=8192,
               sinks=4, lse=True),
        # two prompt chunks that read a cached beginning through a window
        _sinks("sinks_chunk", seqs=2, new=2048, len=16384, q_heads=32, kv_heads=8, dim=128, page=32, window=4096, sinks=16),
        # the state of a beam step: 8 requests of 4 beams of the Nano model reordered, and a page for each one's next token
        _fork("fork_step", requests=8, beams=4, len=1000, q_heads=16, kv_heads=4, dim=64),
        # 16 long prompts opened into 8 beams each
        _fork("fork_prompt", requests=16, beams=8, len=16384, q_heads=32, kv_heads=8, dim=128, page=128, new=4, prompt=True),
        # the pages that a decode batch's windows have left behind, given back and the rest moved together
        _compact("compact_step", seqs=32, len=4096, kv_heads=4, dim=64, window=1024, sinks=4, ended=8),
        # a third of a bf16 cache's requests end, all holes are closed
        _compact("compact_all", seqs=48, len=16384, kv_heads=8, dim=128, bits=16, page=16),
        # the same for large pages of a few sequences, a bounded number of moves
        _compact("compact_some", seqs=7, len=20011, kv_heads=8, dim=128, page=128, ended=2, moves=33),
        # one request's first steps: the smallest call
        _beam("beam_one", requests=1, beams=4, vocab=50257, n_out=8),
        # a step of 32 requests, some beams ended
        _beam("beam_step", requests=32, beams=8, vocab=50257, n_out=16, done=True),
        # wide beams over a large vocabulary, logits in f32
        _beam("beam_wide", requests=16, beams=32, vocab=131071, n_out=64, logits="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    by_name = {c["name"]: c for c in listed()}
    most_bytes, most_flops = work(by_name[LARGEST])["bytes"], work(by_name[WIDEST])["flops"]
    heads = [(16, 4, 64), (32, 8, 128), (64, 8, 128), (8, 8, 64), (12, 2, 128), (16, 1, 128), (9, 3, 64)]

    def one():
        kind = rng.choice(("sinks", "sinks", "fork", "compact", "beam"))
        q_heads, kv_heads, dim = rng.choice(heads)
        page, bits = rng.choice((16, 32, 64, 128)), rng.choice((8, 8, 16))
        if kind == "sinks":
            shape = rng.random()
            new = 1 if shape < 0.4 else _log(rng, 2, 16) if shape < 0.6 else _log(rng, 17, 4096)
            length = max(_log(rng, 1, 131072 if new < 17 else 16384), new)
            return _sinks(None, seqs=_log(rng, 1, 64), new=new, len=length, q_heads=q_heads, kv_heads=kv_heads, dim=dim, bits=bits,
                          page=page, window=_log(rng, 1, length), sinks=rng.choice((0, 1, 4, _log(rng, 1, 2000))),
                          causal=rng.random() < 0.85, lse=rng.random() < 0.5)
        if kind == "fork":
            return _fork(None, requests=_log(rng, 1, 64), beams=_log(rng, 1, 32), len=_log(rng, 1, 16384), q_heads=q_heads,
                         kv_heads=kv_heads, dim=dim, bits=bits, page=page, new=1 if rng.random() < 0.5 else _log(rng, 1, 300),
                         prompt=rng.random() < 0.3)
        if kind == "compact":
            window = rng.choice((0, _log(rng, 1, 4096)))
            return _compact(None, seqs=_log(rng, 1, 64), len=_log(rng, 1, 16384), kv_heads=kv_heads, dim=dim, bits=bits, page=page,
                            window=window, sinks=rng.choice((0, 4, 100)) if window else 0, ended=rng.choice((2, 3, 8)),
                            moves=rng.choice((0, 0, _log(rng, 1, 1000))))
        return _beam(None, requests=_log(rng, 1, 64), beams=_log(rng, 1, 32), vocab=_log(rng, 30, 131072), n_out=_log(rng, 1, 64),
                     logits=rng.choice(("bf16", "f32")), done=rng.random() < 0.5)

    got = None
    while got is None:
        c = one()
        del c["name"]
        w = work(c)
        fits = w["bytes"] <= most_bytes and w["flops"] <= most_flops
        if c["op"] == "sinks":
            rows = c["seqs"] * c["new"]
            fits = fits and rows <= 65536 and rows * c["len"] * c["q_heads"] <= 1 << 31
        elif c["op"] == "beam":
            fits = fits and c["requests"] * c["beams"] * c["vocab"] <= 1 << 26
        else:
            fits = fits and _cache_bytes(c) <= 4 << 30
        if fits:
            got = c
    return got


# ---------------------------------------------------------------- the batch: lengths, rows, pages


def _lens(c):
    """(new rows, length after them) of each sequence: the first has the case's own, the others fewer, odd ones among them."""
    i = np.arange(c["seqs"], dtype=np.int64)
    new = np.maximum(1, c.get("new", 1) - (i * 389) % (c.get("new", 1) // 2 + 1))
    return new, np.maximum(new, c["len"] - (i * 7919) % (c["len"] // 2 + 1))


def _page_bytes(c):
    """Keys and values of a page, with their scales."""
    return 2 * c["kv_heads"] * (c["dim"] * c["page"] * c["bits"] / 8 + (4 if c["bits"] == 8 else 0))


def _slot_bytes(c):
    return 2 * 2 * c["kv_heads"] * c["dim"] * c["page"] * 2.0


def _request_lens(c):
    i = np.arange(c["requests"], dtype=np.int64)
    return np.maximum(1, c["len"] - (i * 7919) % (c["len"] // 2 + 1))


def _fork_blocks(c):
    """Of each request: blocks that all beams share, blocks of a beam, blocks with the new tokens."""
    length = _request_lens(c)
    have = -(-length // c["page"])
    return np.where(c["prompt"], 0, length * 7 // 8 // c["page"]), have, -(-(length + c["new"]) // c["page"])


def _fork_pages(c):
    """Pages that the sequences hold and pages that are free at the start."""
    shared, have, wanted = _fork_blocks(c)
    used = have.sum() if c["prompt"] else (shared + c["beams"] * (have - shared)).sum()
    return int(used), int(c["beams"] * (wanted - have + 1).sum()) + 5


def _cache_bytes(c):
    if c["op"] == "fork":
        return sum(_fork_pages(c)) * _page_bytes(c) + (c["requests"] * c["beams"] + 1) * _slot_bytes(c)
    return int((-(-_lens(c)[1] // c["page"])).sum() * 1.1 + 3) * _page_bytes(c)


def _kept(c, length):
    """Of a sequence's blocks, those that its later rows can see (the window's and the sinks')."""
    b = np.arange(-(-int(length) // c["page"]))
    behind = ((b + 1) * c["page"] <= length - c["window"] + 1) & (b * c["page"] >= c["sinks"])
    return ~behind if c["window"] else np.ones(len(b), bool)


def _ended(c):
    return np.arange(c["seqs"]) % c["ended"] == 1


def work(c):
    if c["op"] == "beam":
        rows = c["requests"] * c["beams"]
        n = float(rows) * c["vocab"]
        return {"bytes": n * (4 if c["logits"] == "f32" else 2) + rows * 9 + c["requests"] * c["n_out"] * 13, "flops": 2 * n}
    if c["op"] == "fork":
        seqs = c["requests"] * c["beams"]
        _, have, wanted = _fork_blocks(c)
        # one row of a page table in and out, the counts of the pages it names; the copies: of every request's beams all but one
        # for a prompt, else those that a draw of parents leaves without a child (the mean of one in e)
        table = float(c["beams"] * (have + wanted).sum()) * 4 * 2 + sum(_fork_pages(c)) * 4
        copies = c["requests"] * (c["beams"] - 1) * (1 if c["prompt"] else 0.37)
        open_part = float(np.mean(_request_lens(c) % c["page"] > 0))
        size = copies * 2 * (_slot_bytes(c) if c["bits"] == 8 else _page_bytes(c) * open_part)
        return {"bytes": table + size, "flops": table / 4 + 4.0 * seqs}
    if c["op"] == "compact":
        _, length = _lens(c)
        pages = -(-length // c["page"])
        n_pages, ended = int(pages.sum() * 1.1) + 3, _ended(c)
        live = sum(0 if e else int(_kept(c, l).sum()) for e, l in zip(ended, length))
        moves = live * (1 - live / n_pages)      # the pages lie at random: so many of the live ones are not among the first
        moves = min(moves, c["moves"]) if c["moves"] else moves
        table = float(pages.sum()) * 8 + n_pages * 12
        return {"bytes": table + moves * 2 * _page_bytes(c), "flops": table / 4}
    new, length = _lens(c)
    rows, row = float(new.sum()), c["kv_heads"] * c["dim"]
    w, s = c["window"], c["sinks"]
    keys = seen = 0.0
    for n, l in zip(new.tolist(), length.tolist()):
        p = np.arange(l - n, l)
        hi = p + 1 if c["causal"] else np.full(n, l)
        lo = np.maximum(0, p + 1 - w)
        keys += float((hi - lo + np.minimum(np.minimum(s, lo), hi)).sum())
        seen += float(l - lo[0] + min(s, int(lo[0])))
    size = 2 * row * seen * c["bits"] / 8 + rows * c["q_heads"] * c["dim"] * 4
    return {"bytes": size, "flops": 4.0 * keys * c["q_heads"] * c["dim"]}


# ---------------------------------------------------------------- inputs


def _ints(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.int32).cuda()


def _cache(c, n_pages, n_slots, gen):
    """A layer's cache, every page of it filled."""
    H, P, D = c["kv_heads"], c["page"], c["dim"]
    s = {}
    for x, shape in (("k", (n_pages, H, P, D)), ("v", (n_pages, H, D, P))):
        values = torch.empty(shape, dtype=torch.int8 if c["bits"] == 8 else torch.bfloat16, device="cuda")
        flat = values.view(-1)
        for a in range(0, flat.numel(), 1 << 28):  # in parts: the normal values are 32 bits wide
            part = flat[a:a + (1 << 28)]
            drawn = torch.randn(part.numel(), generator=gen, device="cuda")
            part.copy_((drawn * 36.0).round_().clamp_(-127, 127) if c["bits"] == 8 else drawn)
        s[x] = values
        if c["bits"] == 8:
            s[x + "_scale"] = torch.rand(n_pages, H, generator=gen, device="cuda") * 0.018 + 0.018
            s[x + "_tail"] = torch.randn(n_slots, 2, *shape[1:], generator=gen, device="cuda").to(torch.bfloat16)
    return s


def _spread(rs, counts, n_pages):
    """A page table with counts[i] pages of its own for row i, spread over the cache at random."""
    table, order, at = np.full((len(counts), int(counts.max())), -1, np.int64), rs.permutation(n_pages), 0
    for i, n in enumerate(counts.tolist()):
        table[i, :n] = order[at:at + n]
        at += n
    return table


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    rs = np.random.RandomState(int(seed) % (1 << 32))
    s = {"case": dict(case)}
    {"sinks": _prepare_sinks, "fork": _prepare_fork, "compact": _prepare_compact, "beam": _prepare_beam}[case["op"]](case, s, gen, rs)
    return s


def _prepare_sinks(c, s, gen, rs):
    new, length = _lens(c)
    S, P = c["seqs"], c["page"]
    per_seq = -(-length // P)
    n_pages = int(per_seq.sum()) + 3
    table = _spread(rs, per_seq, n_pages)
    row_start = np.concatenate([[0], np.cumsum(new)])
    rows = int(row_start[-1])
    s.update(rows=rows, max_rows=int(new.max()), max_len=int(length.max()), n_pages=n_pages, n_slots=S + 1, row_start=_ints(row_start),
             kv_len=_ints(length), pages=_ints(table), slots=_ints(rs.permutation(S + 1)[:S]))
    s.update(_cache(c, n_pages, S + 1, gen))
    s["q"] = (torch.randn(rows, c["q_heads"], c["dim"], generator=gen, device="cuda") * 1.5).to(torch.bfloat16)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(rows, c["q_heads"], device="cuda") if c["lse"] else None


def _fork_tables(c, rs):
    """Page table, lengths and parents before the step: a request's beams share a beginning and have the rest of their own."""
    shared, have, wanted = _fork_blocks(c)
    R, B, width = c["requests"], c["beams"], int(wanted.max())
    used, free = _fork_pages(c)
    order, at = rs.permutation(used + free), 0
    table, lens, parent = np.full((R * B, width), -1, np.int64), np.zeros(R * B, np.int64), np.zeros(R * B, np.int64)
    length = _request_lens(c)
    for r in range(R):
        common, at = order[at:at + shared[r]], at + int(shared[r])
        for b in range(1 if c["prompt"] else B):
            mine = int(have[r] - shared[r])
            table[r * B + b, :shared[r]] = common
            table[r * B + b, shared[r]:have[r]] = order[at:at + mine]
            lens[r * B + b], at = length[r], at + mine
        parent[r * B:(r + 1) * B] = r * B + (0 if c["prompt"] else rs.randint(0, B, B))
    return table, lens, parent, used + free


def _prepare_fork(c, s, gen, rs):
    table, lens, parent, n_pages = _fork_tables(c, rs)
    S = len(lens)
    s.update(n_pages=n_pages, n_slots=S + 1, max_len=int(lens.max()) + c["new"], kv_len=_ints(lens), pages=_ints(table), parent=_ints(parent),
             slots=_ints(rs.permutation(S + 1)[:S]), refs_before=_ints(np.bincount(table[table >= 0], minlength=n_pages)),
             row_start=_ints(np.arange(S + 1) * c["new"]))
    s.update(_cache(c, n_pages, S + 1 if c["bits"] == 8 else 0, gen))
    s.update(refs=torch.empty_like(s["refs_before"]), pages_out=torch.empty_like(s["pages"]))
    for name in ("kv_len_out", "slots_out", "slot_src", "slot_dst", "page_src", "page_dst", "missing"):
        s[name] = torch.empty_like(s["parent"])


def _prepare_compact(c, s, gen, rs):
    _, length = _lens(c)
    per_seq = -(-length // c["page"])
    n_pages = int(per_seq.sum() * 1.1) + 3
    table = _spread(rs, per_seq, n_pages)
    moves = min(c["moves"] or n_pages, n_pages // 2)
    # what a pass changes lies side by side, so that it is put back in one copy
    before = np.concatenate([table.reshape(-1), np.bincount(table[table >= 0], minlength=n_pages)])
    s.update(n_pages=n_pages, n_slots=0, max_len=int(length.max()), before=_ints(before), kv_len=_ints(np.where(_ended(c), 0, length)),
             page_src=_ints(np.zeros(moves)), page_dst=_ints(np.zeros(moves)), n_live=_ints(np.zeros(1)))
    s["now"] = s["before"].clone()
    s["pages"], s["refs"] = s["now"][:table.size].view(table.shape), s["now"][table.size:]
    s.update(_cache(c, n_pages, 0, gen))


def _prepare_beam(c, s, gen, rs):
    R, B, V = c["requests"], c["beams"], c["vocab"]
    logits = torch.randn(R * B, V, generator=gen, device="cuda").mul_(2.5)
    # a few tokens that the program forbids
    logits[:, torch.randint(0, V, (max(1, V // 100),), generator=gen, device="cuda")] = -math.inf
    scores = -torch.rand(R, B, generator=gen, device="cuda") * 6.0 - 20.0
    s.update(logits=logits.to(torch.float32 if c["logits"] == "f32" else torch.bfloat16), scores=scores,
             ended=(torch.rand(R, B, generator=gen, device="cuda") < 0.2) if c["done"] else None, end_token=V // 3)
    n = (R, c["n_out"])
    s.update(parent=torch.empty(n, dtype=torch.int32, device="cuda"), token=torch.empty(n, dtype=torch.int32, device="cuda"),
             score=torch.empty(n, device="cuda"), lse=torch.empty(R, B, device="cuda"),
             ended_out=torch.empty(n, dtype=torch.bool, device="cuda") if c["done"] else None)


# ---------------------------------------------------------------- one pass


def run(state):
    op = state["case"]["op"]
    if own:
        return {"sinks": _own_sinks, "fork": _own_fork, "compact": _own_compact, "beam": _own_beam}[op](state)
    return {"sinks": _plain_sinks, "fork": _plain_fork, "compact": _plain_compact, "beam": _plain_beam}[op](state)


def _handles(state):
    """What a program keeps beside its buffers: the shape, the batch's tables, the cache as the library takes it, workspaces."""
    import int4_routed_expert_02_amd as moe
    c = state["case"]

    def bytes_of(n):
        return torch.empty(n, dtype=torch.uint8, device="cuda")

    if c["op"] == "beam":
        h = (moe, bytes_of(moe.moe_beam_workspace_bytes(c["requests"], c["beams"], c["vocab"], c["n_out"])))
    else:
        cache = moe.kv_cache(state["k"], state["v"], state.get("k_scale"), state.get("v_scale"), state.get("k_tail"), state.get("v_tail"))
        seqs, blocks = state["pages"].shape
        rows = state.get("rows", seqs * c.get("new", 0))
        sh = moe.kv_shape(n_seq=seqs, rows=rows, max_rows=state.get("max_rows", c.get("new", 0)), max_len=state["max_len"],
                          q_heads=c.get("q_heads", c["kv_heads"]), kv_heads=c["kv_heads"], head_dim=c["dim"], kv_bits=c["bits"],
                          page_tokens=c["page"], n_pages=state["n_pages"], max_pages=blocks, n_slots=state["n_slots"],
                          window=c.get("window", 0), flags=0 if c.get("causal", True) else moe.MOE_KV_NONCAUSAL)
        if c["op"] == "sinks":
            batch = moe.kv_batch(state["row_start"], state["kv_len"], state["pages"], state["slots"])
            h = (moe, sh, batch, cache, bytes_of(moe.moe_kv_attention_sinks_workspace_bytes(sh, c["sinks"])))
        elif c["op"] == "fork":
            batch = moe.kv_batch(state["row_start"], state["kv_len"], state["pages"], state["slots"])
            after = moe.kv_batch(state["row_start"], state["kv_len_out"], state["pages_out"], state["slots_out"])
            h = (moe, sh, batch, after, cache, bytes_of(moe.moe_kv_pool_workspace_bytes(sh)))
        else:
            h = (moe, sh, cache, bytes_of(moe.moe_kv_pool_workspace_bytes(sh)))
    state["handles"] = h
    return h


def _own_sinks(s):
    moe, sh, batch, cache, ws = s.get("handles") or _handles(s)
    moe.moe_kv_attention_sinks(sh, s["case"]["sinks"], batch, cache, s["q"], s["out"], s["lse"], ws)
    return {"out": s["out"], "lse": s["lse"]}


def _own_fork(s):
    moe, sh, batch, after, cache, ws = s.get("handles") or _handles(s)
    s["refs"].copy_(s["refs_before"])
    moe.moe_kv_fork(sh, batch, s["parent"], s["kv_len_out"], s["pages_out"], s["slots_out"], s["refs"], s["slot_src"], s["slot_dst"])
    s["kv_len_out"].add_(s["case"]["new"])
    moe.moe_kv_reserve(sh, after, s["pages_out"], s["refs"], s["page_src"], s["page_dst"], s["missing"], ws)
    if s["case"]["bits"] == 8:
        moe.moe_kv_copy(sh, cache, slot_src=s["slot_src"], slot_dst=s["slot_dst"])
    else:
        moe.moe_kv_copy(sh, cache, page_src=s["page_src"], page_dst=s["page_dst"])
    return _forked(s, s["pages_out"], s["refs"], s["kv_len_out"], s["slots_out"], s["missing"])


def _own_compact(s):
    moe, sh, cache, ws = s.get("handles") or _handles(s)
    s["now"].copy_(s["before"])
    moe.moe_kv_release(sh, s["case"]["sinks"], s["kv_len"], s["pages"], s["refs"])
    moe.moe_kv_compact(sh, s["pages"], s["refs"], s["page_src"], s["page_dst"], s["n_live"], ws)
    moe.moe_kv_copy(sh, cache, page_src=s["page_src"], page_dst=s["page_dst"])
    return _compacted(s, s["pages"], s["refs"], s["page_src"], s["page_dst"], s["n_live"])


def _own_beam(s):
    moe, ws = s.get("handles") or _handles(s)
    moe.moe_beam_select(s["logits"], s["scores"], s["parent"], s["token"], s["score"], lse=s["lse"], done=s["ended"], done_out=s["ended_out"],
                        end_token=s["end_token"], ws=ws)
    return {"parent": s["parent"], "token": s["token"], "score": s["score"], "lse": s["lse"], "done": s["ended_out"]}


def _forked(s, pages, refs, kv_len, slots, missing):
    out = {"pages": pages, "refs": refs, "kv_len": kv_len, "missing": missing}
    if s["case"]["bits"] == 8:
        return dict(out, slots=slots, k_tail=s["k_tail"], v_tail=s["v_tail"])
    return dict(out, k=s["k"], v=s["v"])


def _compacted(s, pages, refs, src, dst, n_live):
    out = {"pages": pages, "refs": refs, "src": src, "dst": dst, "n_live": n_live, "k": s["k"], "v": s["v"]}
    return dict(out, k_scale=s["k_scale"], v_scale=s["v_scale"]) if s["case"]["bits"] == 8 else out


def _plain_sinks(state):
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
    pos = ((length - n)[:, None] + i)[..., None]                                               # [S][rows][1]
    seen = (j < length[:, None])[:, None, :] & ((j > pos - c["window"]) | (j < c["sinks"]))
    if c["causal"]:
        seen = seen & (j <= pos)
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


def _move(values, src, dst):
    """values[dst] = values[src] where both are there (-1: no copy)."""
    there = src >= 0
    values[dst[there].long()] = values[src[there].long()]


def _plain_fork(s):
    c = s["case"]
    dev, P, parent = s["k"].device, c["page"], s["parent"].long()
    S, blocks = s["pages"].shape
    n_pages, t, j = s["n_pages"], torch.arange(S, device=dev), torch.arange(blocks, device=dev)
    children = torch.zeros(S, dtype=torch.int64, device=dev).scatter_add_(0, parent, torch.ones_like(parent))
    first = torch.full((S,), S, device=dev).scatter_reduce_(0, parent, t, "amin")
    length = s["kv_len"].long()
    have = (length + P - 1) // P
    # the rows' tables, and how many rows name each page after it
    entry = s["pages"].long()
    named = entry >= 0
    delta = torch.where(j < have[:, None], children[:, None] - 1, -1)
    refs = s["refs_before"].long()
    refs = refs.scatter_add(0, entry.clamp(min=0).flatten(), torch.where(named, delta, 0).flatten())
    pages = torch.where(j < have[parent][:, None], entry[parent], -1)
    # slots: the first of a sequence's continuations keeps its own, the others take those that are left over, in order
    extra, left = first[parent] != t, children == 0
    give, take = torch.argsort((~left).int(), stable=True), torch.argsort((~extra).int(), stable=True)
    slots = s["slots"].long()
    taken = torch.empty_like(slots).scatter_(0, take, slots[give])
    new_slots = torch.where(extra, taken, slots[parent])
    if c["bits"] == 8:
        src = torch.where(extra & (length[parent] > 0), slots[parent], -1)
        _move(s["k_tail"], src, new_slots)
        _move(s["v_tail"], src, new_slots)
    # pages for the new tokens: every block of theirs gets one that no other sequence names
    start = length[parent]
    end = start + c["new"]
    wanted = (j >= (start // P)[:, None]) & (j <= ((end - 1) // P)[:, None])
    named = wanted & (pages >= 0)
    at = pages.clamp(min=0)
    order = t[:, None] * blocks + j
    writers = torch.zeros(n_pages, dtype=torch.int64, device=dev).scatter_add_(0, at.flatten(), named.long().flatten())
    leader = torch.full((n_pages,), S * blocks, device=dev).scatter_reduce_(0, at.flatten(), torch.where(named, order, S * blocks).flatten(), "amin")
    keeps = (refs[at] <= 1) | ((writers[at] == refs[at]) & (leader[at] == order))
    partial = (j == (start // P)[:, None]) & (start % P > 0)[:, None]
    lost = wanted & ~named & partial
    needs = (wanted & ~named & ~partial) | (named & ~keeps)
    rank = needs.flatten().long().cumsum(0).view_as(needs) - 1
    free = torch.argsort((refs > 0).int(), stable=True)
    got = needs & (rank < (refs <= 0).sum())
    page = torch.where(got, free[rank.clamp(min=0, max=n_pages - 1)], -1)
    refs = refs.scatter_add(0, at.flatten(), -(named & needs).long().flatten())
    refs = refs.scatter_add(0, page.clamp(min=0).flatten(), got.long().flatten())
    if c["bits"] == 16:
        copied = got & named & partial
        src, dst = torch.where(copied, pages, -1).amax(1), torch.where(copied, page, -1).amax(1)
        _move(s["k"], src, dst)
        _move(s["v"], src, dst)
    missing = (lost | (needs & ~got)).sum(1)
    pages = torch.where(needs, page, pages)
    return _forked(s, pages.int(), refs.int(), end.int(), new_slots.int(), missing.int())


def _plain_compact(s):
    c = s["case"]
    dev, P, n_pages = s["k"].device, c["page"], s["n_pages"]
    size = s["pages"].shape
    entry, refs = s["before"][:size[0] * size[1]].view(size).long(), s["before"][size[0] * size[1]:].long()
    j, length = torch.arange(size[1], device=dev), s["kv_len"].long()[:, None]
    gone = j * P >= length
    if c["window"]:
        gone = gone | (((j + 1) * P <= length - c["window"] + 1) & (j * P >= c["sinks"]))
    refs = refs.scatter_add(0, entry.clamp(min=0).flatten(), -((entry >= 0) & gone).long().flatten())
    entry = torch.where(gone, -1, entry)
    live = refs > 0
    n_live, p = live.sum(), torch.arange(n_pages, device=dev)
    below = live.long().cumsum(0) - live.long()                   # live pages below each
    hole, mover = ~live & (p < n_live), live & (p >= n_live)
    k = torch.where(hole, p - below, torch.where(mover, n_live - 1 - below, n_pages))
    moves = s["page_src"].numel()
    k = torch.where(k < moves, k, moves)                          # place `moves` takes what is not moved
    src, dst = (torch.full((moves + 1,), -1, device=dev).scatter_(0, torch.where(m, k, moves), torch.where(m, p, -1))[:moves]
                for m in (mover, hole))
    moved = mover & (k < moves)
    to = torch.where(moved, dst[k.clamp(max=moves - 1)], p)
    entry = torch.where(entry >= 0, to[entry.clamp(min=0)], -1)
    after = torch.where(moved, 0, refs)
    after = after.scatter_add(0, to, torch.where(moved, refs, 0))
    for name in ("k", "v", "k_scale", "v_scale") if c["bits"] == 8 else ("k", "v"):
        _move(s[name], src, dst)
    return _compacted(s, entry.int(), after.int(), src.int(), dst.int(), n_live.int()[None])


def _plain_beam(s):
    c = s["case"]
    R, B, n_out = c["requests"], c["beams"], c["n_out"]
    x = s["logits"].double()
    top = x.amax(dim=1, keepdim=True)
    lse = (top + (x - top).exp().sum(dim=1, keepdim=True).log()).view(R, B)
    base = s["scores"].double() - lse
    # a row's own order: the larger logit, then the lower token; of several rows: the larger sum, then the lower row
    value, token = torch.sort(s["logits"], dim=1, descending=True, stable=True)
    n = min(n_out, c["vocab"])
    value, token = value[:, :n].double().view(R, B, n), token[:, :n].view(R, B, n)
    sums = torch.where(torch.isfinite(base)[..., None], base[..., None] + value, -math.inf)
    if s["ended"] is not None:
        at = torch.arange(n, device=x.device)
        stays = torch.where(at == 0, s["scores"].double()[..., None], -math.inf)
        sums = torch.where(s["ended"][..., None], stays, sums)
        token = torch.where(s["ended"][..., None], s["end_token"], token)
    sums, order = torch.sort(sums.flatten(1), dim=1, descending=True, stable=True)
    short = max(0, n_out - B * n)
    sums = torch.nn.functional.pad(sums[:, :n_out], (0, short), value=-math.inf)
    order = torch.nn.functional.pad(order[:, :n_out], (0, short))
    none = sums == -math.inf
    parent = torch.where(none, -1, order // n + torch.arange(R, device=x.device)[:, None] * B)
    token = torch.where(none, -1, token.flatten(1).gather(1, order))
    ended = None
    if s["ended"] is not None:
        ended = none | (token == s["end_token"]) | s["ended"].flatten()[parent.clamp(min=0)]
    return {"parent": parent.int(), "token": token.int(), "score": sums.float(), "lse": lse.float(), "done": ended}


# ---------------------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    return {"sinks": _exact_sinks, "fork": _exact_fork, "compact": _exact_compact, "beam": _exact_beam}[case["op"]](case, prepare(case, seed))


def _exact_sinks(case, s):
    new, length = _lens(case)
    P, H, D, G = case["page"], case["kv_heads"], case["dim"], case["q_heads"] // case["kv_heads"]
    first_row = np.concatenate([[0], np.cumsum(new)]).tolist()
    table, slots = s["pages"].cpu().numpy(), s["slots"].cpu().numpy()
    outs, lses = [], []
    for i in range(case["seqs"]):
        n, l = int(new[i]), int(length[i])
        ids = torch.from_numpy(table[i, :-(-l // P)]).long().cuda()
        q = s["q"][first_row[i]:first_row[i + 1]].double()
        j, p = torch.arange(l, device="cuda"), torch.arange(l - n, l, device="cuda")[:, None]
        hidden = (j <= p - case["window"]) & (j >= case["sinks"])
        if case["causal"]:
            hidden |= j > p
        out = torch.zeros(n, H, G, D, dtype=torch.float64, device="cuda")
        lse = torch.zeros(n, H, G, dtype=torch.float64, device="cuda")
        for h in range(H):
            k, v = s["k"][ids, h].double(), s["v"][ids, h].double().transpose(1, 2)
            if case["bits"] == 8:
                k, v = k * s["k_scale"][ids, h].double()[:, None, None], v * s["v_scale"][ids, h].double()[:, None, None]
                if l % P:
                    k[-1] = s["k_tail"][slots[i], l // P % 2, h].double()
                    v[-1] = s["v_tail"][slots[i], l // P % 2, h].double().t()
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


def _exact_fork(case, s):
    P, new, S = case["page"], case["new"], case["requests"] * case["beams"]
    pages, lens, parent, slots = (s[x].cpu().numpy().tolist() for x in ("pages", "kv_len", "parent", "slots"))
    blocks = len(pages[0])
    out = [[pages[p][b] if b * P < lens[p] else -1 for b in range(blocks)] for p in parent]
    holders = {}
    for row in out:
        for page in row:
            if page >= 0:
                holders[page] = holders.get(page, 0) + 1
    kept = [min((t for t in range(S) if parent[t] == p), default=None) for p in range(S)]
    spare = iter([slots[p] for p in range(S) if kept[p] is None])
    new_slots, copies = [], []
    for t, p in enumerate(parent):
        if kept[p] == t:
            new_slots.append(slots[p])
        else:
            new_slots.append(next(spare))
            if lens[p] > 0:
                copies.append((slots[p], new_slots[-1]))
    span = [(lens[p] // P, (lens[p] + new - 1) // P) for p in parent]
    asked = {}
    for t, (a, b) in enumerate(span):
        for block in range(a, b + 1):
            if out[t][block] >= 0:
                asked.setdefault(out[t][block], []).append((t, block))
    free = iter([p for p in range(s["n_pages"]) if p not in holders])
    missing, moved = [0] * S, []
    before = dict(holders)
    for t, (a, b) in enumerate(span):
        for block in range(a, b + 1):
            page, inside = out[t][block], block == a and lens[parent[t]] % P > 0
            if page >= 0 and (before[page] == 1 or (before[page] == len(asked[page]) and asked[page][0] == (t, block))):
                continue
            if page < 0 and inside:
                missing[t] += 1
                continue
            got = next(free, -1)
            missing[t] += got < 0
            if page >= 0:
                holders[page] -= 1
                if inside and got >= 0:
                    moved.append((page, got))
            if got >= 0:
                holders[got] = 1
            out[t][block] = got
    res = {"pages": torch.tensor(out), "refs": torch.tensor([holders.get(p, 0) for p in range(s["n_pages"])]),
           "kv_len": torch.tensor([lens[p] + new for p in parent]), "missing": torch.tensor(missing)}
    names = ("k_tail", "v_tail") if case["bits"] == 8 else ("k", "v")
    for a, b in copies if case["bits"] == 8 else moved:
        for x in names:
            s[x][b] = s[x][a]
    if case["bits"] == 8:
        res["slots"] = torch.tensor(new_slots)
    return dict(res, **{x: s[x] for x in names})


def _exact_compact(case, s):
    P, n_pages = case["page"], s["n_pages"]
    size = tuple(s["pages"].shape)
    rows = s["before"][:size[0] * size[1]].view(size).cpu().numpy().tolist()
    lens = s["kv_len"].cpu().numpy().tolist()
    for row, l in zip(rows, lens):
        for b in range(len(row)):
            oldest = l - case["window"] + 1                        # the first position in the next row's window
            if b * P >= l or (case["window"] and b * P + P <= oldest and b * P >= case["sinks"]):
                row[b] = -1
    refs = [0] * n_pages
    for row in rows:
        for page in row:
            if page >= 0:
                refs[page] += 1
    n_live, src, dst = sum(r > 0 for r in refs), [], []
    high = [p for p in range(n_pages - 1, n_live - 1, -1) if refs[p]]
    for a, b in list(zip(high, (p for p in range(n_live) if not refs[p])))[:s["page_src"].numel()]:
        src.append(a)
        dst.append(b)
        refs[b], refs[a] = refs[a], 0
    to = dict(zip(src, dst))
    rows = [[to.get(page, page) for page in row] for row in rows]
    names = ("k", "v", "k_scale", "v_scale") if case["bits"] == 8 else ("k", "v")
    for x in names:
        for a, b in to.items():
            s[x][b] = s[x][a]
    pad = [-1] * (s["page_src"].numel() - len(src))
    res = {"pages": torch.tensor(rows), "refs": torch.tensor(refs), "src": torch.tensor(src + pad), "dst": torch.tensor(dst + pad),
           "n_live": torch.tensor([n_live])}
    return dict(res, **{x: s[x] for x in names})


def _exact_beam(case, s):
    B, V, n_out = case["beams"], case["vocab"], case["n_out"]
    parents, tokens, scores, lses, ends = [], [], [], [], []
    for r in range(case["requests"]):
        x = s["logits"][r * B:(r + 1) * B].double()
        lse = torch.logsumexp(x, dim=1)
        sums = x + (s["scores"][r].double() - lse)[:, None]
        sums[torch.isnan(sums)] = -math.inf
        if s["ended"] is not None:
            for b in torch.nonzero(s["ended"][r]).flatten().tolist():
                sums[b] = -math.inf
                sums[b, s["end_token"]] = s["scores"][r, b].double()
        value, at = torch.sort(sums.flatten(), descending=True, stable=True)
        value, at = value[:n_out], at[:n_out]
        pad = n_out - value.numel()
        value, at = torch.nn.functional.pad(value, (0, pad), value=-math.inf), torch.nn.functional.pad(at, (0, pad))
        none = torch.isneginf(value)
        row, token = at // V, torch.where(none, -1, at % V)
        parents.append(torch.where(none, -1, row + r * B))
        tokens.append(token)
        scores.append(value)
        lses.append(lse)
        if s["ended"] is not None:
            ends.append(none | (token == s["end_token"]) | s["ended"][r][row])
    return {"parent": torch.stack(parents), "token": torch.stack(tokens), "score": torch.stack(scores), "lse": torch.stack(lses),
            "done": torch.stack(ends) if ends else None}


if __name__ == "__main__":
    for each in listed() + [draw(random.Random(n)) for n in range(8)]:
        print(each, work(each))
