"""Python binding of the MI355X MoE-layer library (libmoe_hip.so, include/moe.h).

Argument marshalling only: every step of the layer runs in the library's HIP
kernels.  torch provides device memory and the current stream.  If the HIP
library is missing, every call raises -- there is no CPU fallback.

The functions mirror the C ABI names:
  moe_router, moe_permute, moe_expert_ffn, moe_combine, moe_layer_forward,
  moe_workspace_bytes, moe_validate_shape, moe_status_string, moe_layer_routing,
  moe_quantize_rows, moe_bias_update, moe_layer_forward_chain, moe_quantize_act_q8,
  moe_kv_append, moe_kv_attention, moe_kv_read, moe_kv_workspace_bytes,
  moe_linear_q4, moe_linear_q4_workspace_bytes, moe_kv_attention_sinks,
  moe_kv_attention_sinks_workspace_bytes, moe_kv_release, moe_kv_fork, moe_kv_reserve,
  moe_kv_compact, moe_kv_copy, moe_kv_pool_workspace_bytes, moe_beam_select,
  moe_beam_workspace_bytes
and ``MoeLayer`` keeps one layer's device weights and workspace, ``KvPages`` one
layer's key/value cache.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmoe_hip.so")

MOE_OK = 0
MOE_ERR_NULL = -1
MOE_ERR_SHAPE = -2
MOE_ERR_UNSUPPORTED = -3
MOE_ERR_WORKSPACE = -4
MOE_ERR_ALIGN = -5
MOE_ERR_HIP = -6

MOE_OUT_F32 = 1
MOE_ADD_RESIDUAL = 2
MOE_EXPERT_INT8 = 4
MOE_TEST_GATEUP_SUMS = 0x100
MOE_STAGE_GATEUP_ONLY = 0x200
MOE_STAGE_EXPERTS_ONLY = 0x400
MOE_LOGITS_GIVEN = 0x800
MOE_ACT_Q8 = 0x1000
MOE_EXPERT_MIXED = 0x2000
MOE_REGIME_TILED = 0x4000
MOE_REGIME_SMALL = 0x8000

MOE_KV_NONCAUSAL = 0x10000
MOE_KV_ROPE_PAIRS = 0x20000

MOE_SRC_F32 = 0
MOE_SRC_BF16 = 1

MOE_WS_PERMUTE = 1
MOE_WS_EXPERT_FFN = 2
MOE_WS_LAYER = 3

EXPORTS = ["moe_router", "moe_permute", "moe_expert_ffn", "moe_combine", "moe_layer_forward",
           "moe_layer_forward_profiled", "moe_workspace_bytes", "moe_validate_shape", "moe_status_string",
           "moe_layer_routing", "moe_quantize_rows", "moe_bias_update", "moe_layer_forward_chain",
           "moe_quantize_act_q8", "moe_layer_forward_noalloc", "moe_kv_append", "moe_kv_attention", "moe_kv_read",
           "moe_kv_workspace_bytes", "moe_linear_q4", "moe_linear_q4_workspace_bytes", "moe_kv_attention_sinks",
           "moe_kv_attention_sinks_workspace_bytes", "moe_kv_release", "moe_kv_fork", "moe_kv_reserve", "moe_kv_compact",
           "moe_kv_copy", "moe_kv_pool_workspace_bytes", "moe_beam_select", "moe_beam_workspace_bytes"]

MOE_NOALLOC_SCRATCH_BYTES = 64 << 20
MOE_KV_FORK_MAX = 8192


class MoeShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("E", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("I", ctypes.c_int32), ("I_shared", ctypes.c_int32),
                ("shared_bits", ctypes.c_int32), ("n_group", ctypes.c_int32),
                ("topk_group", ctypes.c_int32), ("routed_scaling_factor", ctypes.c_float),
                ("flags", ctypes.c_uint32), ("top_p", ctypes.c_float)]


class MoeQMat(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("qs", ctypes.c_void_p),
                ("q_stride_bytes", ctypes.c_int64), ("qs_stride_floats", ctypes.c_int64)]


class MoeWeights(ctypes.Structure):
    _fields_ = [("router_w", ctypes.c_void_p), ("router_bias", ctypes.c_void_p),
                ("gate", MoeQMat), ("up", MoeQMat), ("down", MoeQMat),
                ("sh_gate", MoeQMat), ("sh_up", MoeQMat), ("sh_down", MoeQMat), ("expert_bits", ctypes.c_void_p)]


class MoeKvShape(ctypes.Structure):
    _fields_ = [("n_seq", ctypes.c_int32), ("rows", ctypes.c_int32), ("max_rows", ctypes.c_int32),
                ("max_len", ctypes.c_int32), ("q_heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("kv_bits", ctypes.c_int32), ("page_tokens", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("n_slots", ctypes.c_int32),
                ("window", ctypes.c_int32), ("scale", ctypes.c_float), ("flags", ctypes.c_uint32)]


class MoeKvBatch(ctypes.Structure):
    _fields_ = [("row_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("pages", ctypes.c_void_p),
                ("slots", ctypes.c_void_p)]


class MoeKvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("k_tail", ctypes.c_void_p), ("v_tail", ctypes.c_void_p)]


class MoeKvRotary(ctypes.Structure):
    _fields_ = [("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("n_pos", ctypes.c_int32),
                ("rot_dim", ctypes.c_int32), ("pos", ctypes.c_void_p), ("q_norm", ctypes.c_void_p),
                ("k_norm", ctypes.c_void_p), ("eps", ctypes.c_float)]


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} ({status})")
        self.status = status


_lib = None


def load() -> ctypes.CDLL:
    """Load libmoe_hip.so; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                              "(hipcc --offload-arch=gfx950); there is no fallback path")
        L = ctypes.CDLL(LIB_PATH)
        vp, S, W = ctypes.c_void_p, ctypes.POINTER(MoeShape), ctypes.POINTER(MoeWeights)
        sz, i32, i64 = ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64
        KS, KB, KC = ctypes.POINTER(MoeKvShape), ctypes.POINTER(MoeKvBatch), ctypes.POINTER(MoeKvCache)
        sig = {
            "moe_router": [S, vp, vp, vp, vp, vp, vp, vp, sz, vp],
            "moe_permute": [S, vp, vp, vp, vp, vp, vp, sz, vp],
            "moe_expert_ffn": [S, vp, W, vp, vp, vp, vp, vp, sz, vp],
            "moe_combine": [S, vp, vp, vp, vp, vp, vp, vp],
            "moe_layer_forward": [S, W, vp, vp, vp, sz, vp],
            "moe_layer_forward_profiled": [S, W, vp, vp, vp, sz, vp, vp, vp],
            "moe_layer_forward_noalloc": [S, W, vp, vp, vp],
            "moe_layer_forward_chain": [S, W, vp, vp, vp, sz, S, W, vp, sz, vp],
            "moe_validate_shape": [S],
            "moe_layer_routing": [S, vp, sz, vp, vp, vp, vp],
            "moe_quantize_rows": [vp, ctypes.c_int32, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, vp, vp, vp],
            "moe_quantize_act_q8": [vp, ctypes.c_int32, ctypes.c_int64, ctypes.c_int32, vp, vp, vp],
            "moe_bias_update": [ctypes.c_int32, vp, vp, ctypes.c_float, vp],
            "moe_kv_append": [KS, KB, KC, ctypes.POINTER(MoeKvRotary), vp, i64, vp, i64, vp, i64, vp, vp],
            "moe_kv_attention": [KS, KB, KC, vp, i64, vp, vp, vp, sz, vp],
            "moe_kv_read": [KS, KB, KC, vp, vp, vp],
            "moe_linear_q4": [i32, i32, i32, i32, vp, i64, vp, vp, i32, vp, vp, ctypes.c_uint32, vp, sz, vp],
            "moe_kv_attention_sinks": [KS, i32, KB, KC, vp, i64, vp, vp, vp, sz, vp],
            "moe_kv_release": [KS, i32, vp, vp, vp, vp],
            "moe_kv_fork": [KS, KB, vp, vp, vp, vp, vp, vp, vp, vp],
            "moe_kv_reserve": [KS, KB, vp, vp, vp, vp, vp, vp, sz, vp],
            "moe_kv_compact": [KS, vp, vp, i32, vp, vp, vp, vp, sz, vp],
            "moe_kv_copy": [KS, KC, i32, vp, vp, i32, vp, vp, vp],
            "moe_beam_select": [i32, i32, i32, i32, vp, i32, i64, vp, vp, i32, vp, vp, vp, vp, vp, vp, sz, vp],
        }
        for name, args in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        L.moe_workspace_bytes.argtypes = [S, ctypes.c_int]
        L.moe_workspace_bytes.restype = ctypes.c_size_t
        L.moe_kv_workspace_bytes.argtypes = [KS]
        L.moe_kv_workspace_bytes.restype = sz
        L.moe_linear_q4_workspace_bytes.argtypes = [i32, i32, i32]
        L.moe_linear_q4_workspace_bytes.restype = sz
        L.moe_kv_attention_sinks_workspace_bytes.argtypes = [KS, i32]
        L.moe_kv_attention_sinks_workspace_bytes.restype = sz
        L.moe_kv_pool_workspace_bytes.argtypes = [KS]
        L.moe_kv_pool_workspace_bytes.restype = sz
        L.moe_beam_workspace_bytes.argtypes = [i32, i32, i32, i32]
        L.moe_beam_workspace_bytes.restype = sz
        L.moe_status_string.argtypes = [ctypes.c_int]
        L.moe_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return load().moe_status_string(status).decode()


moe_status_string = status_string


def _check(status: int, what: str):
    if status != MOE_OK:
        raise MoeError(status, what)


def shape(T, H, E, top_k, I, I_shared=0, shared_bits=0, n_group=1, topk_group=1, rsf=1.0, flags=0,
          top_p=0.0) -> MoeShape:
    return MoeShape(T, H, E, top_k, I, I_shared, shared_bits, n_group, topk_group, rsf, flags, top_p)


def shape_of(cfg, T: Optional[int] = None, flags: int = 0) -> MoeShape:
    """MoeShape of a synth.LayerConfig-like object (fields T,H,E,k,I,I_sh,...)."""
    if getattr(cfg, "act_q8", False):
        flags |= MOE_ACT_Q8
    if getattr(cfg, "int2_frac", 0.0) > 0:
        flags |= MOE_EXPERT_MIXED
    return shape(cfg.T if T is None else T, cfg.H, cfg.E, cfg.k, cfg.I, cfg.I_sh, cfg.shared_bits, cfg.n_group,
                 cfg.topk_group, cfg.rsf, flags, float(getattr(cfg, "top_p", 0.0)))


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must be on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


# torch, once a call has needed it, the current stream's handle as torch keeps it, and the tables' type
_torch = _current = _int32 = None


def _bind_torch():
    """torch is imported by the first call that needs it, not with the package."""
    global _torch, _current, _int32
    import torch
    _torch, _int32 = torch, torch.int32
    get_device = getattr(torch._C, "_cuda_getDevice", None)
    raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if get_device is not None and raw_stream is not None:
        # a tenth of a microsecond; torch.cuda.current_stream() builds an object, 3 us
        _current = lambda: raw_stream(get_device())  # noqa: E731
    else:
        _current = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    return torch


def _stream(stream) -> Optional[int]:
    if stream is not None:
        return stream.cuda_stream
    if _current is None:
        _bind_torch()
    return _current()


def moe_validate_shape(sh: MoeShape) -> int:
    return load().moe_validate_shape(ctypes.byref(sh))


def moe_workspace_bytes(sh: MoeShape, which: int = MOE_WS_LAYER) -> int:
    return int(load().moe_workspace_bytes(ctypes.byref(sh), which))


def moe_router(sh: MoeShape, hidden, router_w, router_bias, topk_ids, topk_w, sel_gap, ws, stream=None):
    _check(load().moe_router(ctypes.byref(sh), _ptr(hidden), _ptr(router_w), _ptr(router_bias), _ptr(topk_ids),
                             _ptr(topk_w), _ptr(sel_gap), _ptr(ws), ws.numel() if ws is not None else 0,
                             _stream(stream)), "moe_router")


def moe_permute(sh: MoeShape, topk_ids, counts, offsets, sorted_pairs, inv_pos, ws, stream=None):
    _check(load().moe_permute(ctypes.byref(sh), _ptr(topk_ids), _ptr(counts), _ptr(offsets), _ptr(sorted_pairs),
                              _ptr(inv_pos), _ptr(ws), ws.numel() if ws is not None else 0, _stream(stream)),
           "moe_permute")


def moe_expert_ffn(sh: MoeShape, hidden, weights: MoeWeights, offsets, sorted_pairs, pair_scale, y_pairs, ws,
                   stream=None):
    _check(load().moe_expert_ffn(ctypes.byref(sh), _ptr(hidden), ctypes.byref(weights), _ptr(offsets),
                                 _ptr(sorted_pairs), _ptr(pair_scale), _ptr(y_pairs), _ptr(ws),
                                 ws.numel() if ws is not None else 0, _stream(stream)), "moe_expert_ffn")


def moe_combine(sh: MoeShape, y_pairs, inv_pos, topk_w, shared_out, residual, out, stream=None):
    _check(load().moe_combine(ctypes.byref(sh), _ptr(y_pairs), _ptr(inv_pos), _ptr(topk_w), _ptr(shared_out),
                              _ptr(residual), _ptr(out), _stream(stream)), "moe_combine")


def moe_layer_forward(sh: MoeShape, weights: MoeWeights, hidden, out, ws, stream=None):
    _check(load().moe_layer_forward(ctypes.byref(sh), ctypes.byref(weights), _ptr(hidden), _ptr(out), _ptr(ws),
                                    ws.numel() if ws is not None else 0, _stream(stream)), "moe_layer_forward")


def moe_layer_forward_profiled(sh: MoeShape, weights: MoeWeights, hidden, out, ws, ev_start, ev_stop, stream=None):
    """moe_layer_forward with torch.cuda.Event objects recorded around the expert gate/up kernel."""
    _check(load().moe_layer_forward_profiled(ctypes.byref(sh), ctypes.byref(weights), _ptr(hidden), _ptr(out),
                                             _ptr(ws), ws.numel() if ws is not None else 0, _stream(stream),
                                             ev_start.cuda_event, ev_stop.cuda_event), "moe_layer_forward_profiled")


def moe_layer_forward_noalloc(sh: MoeShape, weights: MoeWeights, hidden, out, stream=None):
    """moe_layer_forward on the library's static scratch: no workspace, no allocation (include/moe.h)."""
    _check(load().moe_layer_forward_noalloc(ctypes.byref(sh), ctypes.byref(weights), _ptr(hidden), _ptr(out),
                                            _stream(stream)), "moe_layer_forward_noalloc")


def moe_layer_forward_chain(sh: MoeShape, weights: MoeWeights, hidden, out, ws, next_sh: Optional[MoeShape] = None,
                            next_weights: Optional[MoeWeights] = None, next_ws=None, stream=None):
    """One layer of a chained small-batch decode step (include/moe.h)."""
    _check(load().moe_layer_forward_chain(ctypes.byref(sh), ctypes.byref(weights), _ptr(hidden), _ptr(out), _ptr(ws),
                                          ws.numel(), ctypes.byref(next_sh) if next_sh is not None else None,
                                          ctypes.byref(next_weights) if next_weights is not None else None,
                                          _ptr(next_ws), next_ws.numel() if next_ws is not None else 0,
                                          _stream(stream)), "moe_layer_forward_chain")


def moe_layer_routing(sh: MoeShape, ws):
    """Device pointers (ints) of ids, w, offsets, sorted inside a layer workspace."""
    p = [ctypes.c_void_p() for _ in range(4)]
    _check(load().moe_layer_routing(ctypes.byref(sh), _ptr(ws), ws.numel(), *[ctypes.byref(x) for x in p]),
           "moe_layer_routing")
    return [x.value for x in p]


def moe_quantize_rows(src, bits: int, q=None, qs=None, stream=None):
    """Per-row symmetric quantiser (include/moe.h): src a 2-D float32 or
    bfloat16 GPU tensor.  Allocates the outputs when not given and returns
    (q, qs): q uint8 [rows][cols/2] (packed int4) or int8 [rows][cols], qs
    float32 [rows]."""
    import torch
    if src.dim() != 2 or src.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("src must be a 2-D float32 or bfloat16 tensor")
    rows, cols = src.shape
    if q is None:
        q = torch.empty((rows, cols // 2) if bits == 4 else (rows, cols),
                        dtype=torch.uint8 if bits == 4 else torch.int8, device=src.device)
    if qs is None:
        qs = torch.empty(rows, dtype=torch.float32, device=src.device)
    fmt = MOE_SRC_BF16 if src.dtype == torch.bfloat16 else MOE_SRC_F32
    _check(load().moe_quantize_rows(_ptr(src), fmt, rows, cols, bits, _ptr(q), _ptr(qs), _stream(stream)),
           "moe_quantize_rows")
    return q, qs


def moe_quantize_act_q8(src, q=None, d=None, stream=None):
    """Q8_0-style activation codes (include/moe.h): src a 2-D float32 or
    bfloat16 GPU tensor with cols % 32 == 0.  Returns (q int8 [rows][cols],
    d float32 [rows][cols/32]), allocated when not given."""
    import torch
    if src.dim() != 2 or src.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("src must be a 2-D float32 or bfloat16 tensor")
    rows, cols = src.shape
    if q is None:
        q = torch.empty((rows, cols), dtype=torch.int8, device=src.device)
    if d is None:
        d = torch.empty((rows, max(cols // 32, 1)), dtype=torch.float32, device=src.device)
    fmt = MOE_SRC_BF16 if src.dtype == torch.bfloat16 else MOE_SRC_F32
    _check(load().moe_quantize_act_q8(_ptr(src), fmt, rows, cols, _ptr(q), _ptr(d), _stream(stream)),
           "moe_quantize_act_q8")
    return q, d


def moe_bias_update(counts, router_bias, gamma: float, stream=None):
    """Aux-loss-free balancing step (include/moe.h): router_bias (f32 [E], GPU)
    is updated in place from counts (int32 [E], GPU)."""
    if counts.numel() != router_bias.numel():
        raise ValueError("counts and router_bias must both have E elements")
    _check(load().moe_bias_update(router_bias.numel(), _ptr(counts), _ptr(router_bias), gamma, _stream(stream)),
           "moe_bias_update")


# ---- the rest of a decoder layer: projections, cache, attention (include/moe.h)


def kv_shape(n_seq, rows, max_rows, max_len, q_heads, kv_heads, head_dim, kv_bits=8, page_tokens=64, n_pages=0,
             max_pages=0, n_slots=0, window=0, scale=0.0, flags=0) -> MoeKvShape:
    return MoeKvShape(n_seq, rows, max_rows, max_len, q_heads, kv_heads, head_dim, kv_bits, page_tokens, n_pages,
                      max_pages, n_slots, window, scale, flags)


def _typed(t, dtype, what):
    if t is not None and t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype}")
    return _ptr(t)


def kv_batch(row_start, kv_len, pages, slots=None) -> MoeKvBatch:
    """The batch's device tables (int32): row_start [n_seq + 1], kv_len [n_seq], pages [n_seq][max_pages], slots
    [n_seq] or None.  The struct keeps the tensors alive."""
    import torch
    b = MoeKvBatch(*(_typed(t, torch.int32, "the batch's tables") for t in (row_start, kv_len, pages, slots)))
    b.tensors = (row_start, kv_len, pages, slots)
    b.sizes = (row_start.numel(), kv_len.numel(), tuple(pages.shape), slots.numel() if slots is not None else None)
    return b


def kv_cache(k, v, k_scale=None, v_scale=None, k_tail=None, v_tail=None) -> MoeKvCache:
    """One layer's cache tensors: int8 codes with f32 scales and bf16 open pages, or bf16 k and v alone.  The struct
    keeps the tensors alive."""
    import torch
    codes = torch.int8 if k_scale is not None else torch.bfloat16
    c = MoeKvCache(_typed(k, codes, "k"), _typed(v, codes, "v"), _typed(k_scale, torch.float32, "k_scale"),
                   _typed(v_scale, torch.float32, "v_scale"), _typed(k_tail, torch.bfloat16, "k_tail"),
                   _typed(v_tail, torch.bfloat16, "v_tail"))
    c.tensors = (k, v, k_scale, v_scale, k_tail, v_tail)
    c.sizes = tuple(tuple(t.shape) if t is not None else None for t in c.tensors)
    return c


def _kv_fits(sh, batch, cache):
    """The tensors are as large as the shape says (the library sees only their addresses)."""
    n, pages = sh.n_seq, (sh.n_seq, sh.max_pages)
    starts, lens, table, slots = batch.sizes
    if starts < n + 1 or lens < n or table != pages or (slots is not None and slots < n):
        raise ValueError("the batch's tables do not fit the shape")
    if sh.kv_bits == 8 and slots is None and sh.n_slots < n:
        raise ValueError("n_slots is below n_seq and no slots are given")
    if cache.sizes != _cache_sizes(sh):
        raise ValueError("the cache's tensors do not fit the shape")


def _cache_sizes(sh):
    h, p, d = sh.kv_heads, sh.page_tokens, sh.head_dim
    sizes = ((sh.n_pages, h, p, d), (sh.n_pages, h, d, p))
    if sh.kv_bits == 8:
        return sizes + ((sh.n_pages, h), (sh.n_pages, h), (sh.n_slots, 2, h, p, d), (sh.n_slots, 2, h, d, p))
    return sizes + (None,) * 4


def kv_rotary(cos=None, sin=None, rot_dim=0, pos=None, q_norm=None, k_norm=None, eps=1e-6) -> MoeKvRotary:
    """Position tables cos and sin [n_pos][rot_dim / 2] (f32), positions pos [rows] (int32) or None for the cache's
    own, and the per-head norm weights (f32 [head_dim]) of q and k, each or None."""
    import torch
    for t in (cos, sin):
        if rot_dim and (t is None or t.dim() != 2 or t.shape != cos.shape or t.shape[1] * 2 != rot_dim):
            raise ValueError("cos and sin must be [n_pos][rot_dim / 2]")
    r = MoeKvRotary(_typed(cos, torch.float32, "cos"), _typed(sin, torch.float32, "sin"),
                    cos.shape[0] if cos is not None else 0, rot_dim, _typed(pos, torch.int32, "pos"),
                    _typed(q_norm, torch.float32, "q_norm"), _typed(k_norm, torch.float32, "k_norm"), eps)
    r.tensors = (cos, sin, pos, q_norm, k_norm)
    r.sizes = tuple(t.numel() if t is not None else None for t in (pos, q_norm, k_norm))
    return r


def _head_rows(t, rows, heads, dim, what):
    """Pointer and row stride of a [rows][heads][dim] bf16 tensor whose rows may be apart."""
    torch = _torch or _bind_torch()
    if t.dtype is not torch.bfloat16 or not t.is_cuda:
        raise ValueError(f"{what} must be a bfloat16 GPU tensor")
    stride = t.stride()
    if t.shape != (rows, heads, dim):
        raise ValueError(f"{what} must be [{rows}][{heads}][{dim}]")
    if rows and (stride[2] != 1 or (heads > 1 and stride[1] != dim)):
        raise ValueError(f"{what}: the heads of a row must be contiguous")
    return t.data_ptr(), stride[0] if rows > 1 else heads * dim


def _head_out(t, rows, heads, dim, what, f32=False):
    torch = _torch or _bind_torch()
    if t.dtype is not (torch.float32 if f32 else torch.bfloat16) or t.shape != (rows, heads, dim):
        raise ValueError(f"{what} must be a {'float32' if f32 else 'bfloat16'} [{rows}][{heads}][{dim}] tensor")
    return _ptr(t)


def moe_kv_workspace_bytes(sh: MoeKvShape) -> int:
    return int(load().moe_kv_workspace_bytes(ctypes.byref(sh)))


def moe_kv_append(sh: MoeKvShape, batch: MoeKvBatch, cache: MoeKvCache, k, v, rot: Optional[MoeKvRotary] = None,
                  q=None, q_out=None, stream=None):
    """Store the batch's keys and values (norm and rotation of k on the way) and rotate q into q_out (include/moe.h).
    k, v [rows][kv_heads][head_dim] and q [rows][q_heads][head_dim] bf16, rows possibly apart."""
    _kv_fits(sh, batch, cache)
    if rot is not None and (rot.sizes[0] not in (None, sh.rows) or rot.sizes[1] not in (None, sh.head_dim) or
                            rot.sizes[2] not in (None, sh.head_dim)):
        raise ValueError("pos must be [rows], q_norm and k_norm [head_dim]")
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out come together")
    kp, ks = _head_rows(k, sh.rows, sh.kv_heads, sh.head_dim, "k")
    vp, vs = _head_rows(v, sh.rows, sh.kv_heads, sh.head_dim, "v")
    qp, qs = _head_rows(q, sh.rows, sh.q_heads, sh.head_dim, "q") if q is not None else (None, 0)
    qo = _head_out(q_out, sh.rows, sh.q_heads, sh.head_dim, "q_out") if q_out is not None else None
    _check(load().moe_kv_append(sh, batch, cache, rot, kp, ks, vp, vs, qp, qs, qo, _stream(stream)), "moe_kv_append")


def moe_kv_attention(sh: MoeKvShape, batch: MoeKvBatch, cache: MoeKvCache, q, out, lse=None, ws=None, stream=None):
    """Attention of the batch's rows over the cache (include/moe.h): out [rows][q_heads][head_dim] (bf16, or f32 with
    MOE_OUT_F32), lse [rows][q_heads] f32 or None, ws moe_kv_workspace_bytes(sh) bytes."""
    _check(load().moe_kv_attention(sh, batch, cache, *_attention_args(sh, batch, cache, q, out, lse, ws), _stream(stream)),
           "moe_kv_attention")


def _attention_args(sh, batch, cache, q, out, lse, ws):
    torch = _torch or _bind_torch()
    _kv_fits(sh, batch, cache)
    qp, qs = _head_rows(q, sh.rows, sh.q_heads, sh.head_dim, "q")
    op = _head_out(out, sh.rows, sh.q_heads, sh.head_dim, "out", bool(sh.flags & MOE_OUT_F32))
    if lse is not None and lse.numel() != sh.rows * sh.q_heads:
        raise ValueError("lse must be [rows][q_heads]")
    return qp, qs, op, _typed(lse, torch.float32, "lse"), _ptr(ws), ws.numel() if ws is not None else 0


def moe_kv_attention_sinks_workspace_bytes(sh: MoeKvShape, sink_tokens: int) -> int:
    return int(load().moe_kv_attention_sinks_workspace_bytes(ctypes.byref(sh), sink_tokens))


def moe_kv_attention_sinks(sh: MoeKvShape, sink_tokens: int, batch: MoeKvBatch, cache: MoeKvCache, q, out, lse=None, ws=None,
                           stream=None):
    """moe_kv_attention where the first sink_tokens positions stay visible behind the shape's window (include/moe.h); ws
    moe_kv_attention_sinks_workspace_bytes(sh, sink_tokens) bytes."""
    _check(load().moe_kv_attention_sinks(sh, sink_tokens, batch, cache, *_attention_args(sh, batch, cache, q, out, lse, ws),
                                         _stream(stream)), "moe_kv_attention_sinks")


def moe_kv_read(sh: MoeKvShape, batch: MoeKvBatch, cache: MoeKvCache, k, v, stream=None):
    """The stored values of the batch's rows (include/moe.h) into k, v [rows][kv_heads][head_dim] bf16."""
    _kv_fits(sh, batch, cache)
    kp = _head_out(k, sh.rows, sh.kv_heads, sh.head_dim, "k")
    vp = _head_out(v, sh.rows, sh.kv_heads, sh.head_dim, "v")
    _check(load().moe_kv_read(sh, batch, cache, kp, vp, _stream(stream)), "moe_kv_read")


# ---- the cache's pages (include/moe.h): tables and counts on the device


def _ints(t, n, what):
    """Pointer of an int32 GPU tensor with n elements (None stays None)."""
    if t is None:
        return None
    if _int32 is None:
        _bind_torch()
    if t.dtype is _int32 and t.numel() == n and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{what} must be a contiguous int32 GPU tensor with {n} elements")


def moe_kv_pool_workspace_bytes(sh: MoeKvShape) -> int:
    return int(load().moe_kv_pool_workspace_bytes(ctypes.byref(sh)))


def moe_kv_release(sh: MoeKvShape, sink_tokens: int, kv_len, pages, refs, stream=None):
    """Give back the pages behind kv_len [n_seq] and those between the sinks and the shape's window (include/moe.h);
    pages [n_seq][max_pages] and refs [n_pages] are changed in place."""
    n = sh.n_seq
    _check(load().moe_kv_release(sh, sink_tokens, _ints(kv_len, n, "kv_len"), _ints(pages, n * sh.max_pages, "pages"),
                                 _ints(refs, sh.n_pages, "refs"), _stream(stream)), "moe_kv_release")


def moe_kv_fork(sh: MoeKvShape, batch: MoeKvBatch, parent, kv_len, pages, slots, refs, slot_src=None, slot_dst=None,
                stream=None):
    """Sequence s goes on from parent[s] (include/moe.h): the batch's state before, kv_len, pages, slots and the lists of
    open pages to copy (slot_src, slot_dst) after; refs is changed in place.  slots and the lists may be None in 16 bits."""
    n, blocks = sh.n_seq, sh.max_pages
    _, lens, table, slots_in = batch.sizes
    if lens < n or table != (n, blocks) or (slots_in is not None and slots_in < n):
        raise ValueError("the batch's tables do not fit the shape")
    _check(load().moe_kv_fork(sh, batch, _ints(parent, n, "parent"), _ints(kv_len, n, "kv_len"), _ints(pages, n * blocks, "pages"),
                              _ints(slots, n, "slots"), _ints(refs, sh.n_pages, "refs"), _ints(slot_src, n, "slot_src"),
                              _ints(slot_dst, n, "slot_dst"), _stream(stream)), "moe_kv_fork")


def moe_kv_reserve(sh: MoeKvShape, batch: MoeKvBatch, pages, refs, copy_src=None, copy_dst=None, missing=None, ws=None,
                   stream=None):
    """Pages of their own for the batch's coming rows (include/moe.h), in place in pages (the batch's table, as a rule)
    and refs; copy_src, copy_dst [n_seq] (16 bits): the pages to copy before the append; missing [n_seq] or None; ws
    moe_kv_pool_workspace_bytes(sh) bytes."""
    n = sh.n_seq
    if batch.sizes[0] < n + 1 or batch.sizes[1] < n:
        raise ValueError("the batch's tables do not fit the shape")
    _check(load().moe_kv_reserve(sh, batch, _ints(pages, n * sh.max_pages, "pages"), _ints(refs, sh.n_pages, "refs"),
                                 _ints(copy_src, n, "copy_src"), _ints(copy_dst, n, "copy_dst"), _ints(missing, n, "missing"), _ptr(ws),
                                 ws.numel() if ws is not None else 0, _stream(stream)), "moe_kv_reserve")


def moe_kv_compact(sh: MoeKvShape, pages, refs, copy_src, copy_dst, n_live=None, ws=None, stream=None):
    """Move the pages in use to the lowest ids, as many as copy_src and copy_dst have room for (include/moe.h; None: no moves);
    pages and refs are changed in place, n_live [1] or None."""
    if (copy_src is None) != (copy_dst is None):
        raise ValueError("a list's sources and destinations come together")
    moves = copy_src.numel() if copy_src is not None else 0
    _check(load().moe_kv_compact(sh, _ints(pages, sh.n_seq * sh.max_pages, "pages"), _ints(refs, sh.n_pages, "refs"), moves,
                                 _ints(copy_src, moves, "copy_src"), _ints(copy_dst, moves, "copy_dst"), _ints(n_live, 1, "n_live"),
                                 _ptr(ws), ws.numel() if ws is not None else 0, _stream(stream)), "moe_kv_compact")


def moe_kv_copy(sh: MoeKvShape, cache: MoeKvCache, page_src=None, page_dst=None, slot_src=None, slot_dst=None, stream=None):
    """Copy pages and open pages of one layer's cache by the lists of the calls above (include/moe.h)."""
    if cache.sizes != _cache_sizes(sh):
        raise ValueError("the cache's tensors do not fit the shape")
    if (page_src is None) != (page_dst is None) or (slot_src is None) != (slot_dst is None):
        raise ValueError("a list's sources and destinations come together")
    pages, slots = (t.numel() if t is not None else 0 for t in (page_src, slot_src))
    _check(load().moe_kv_copy(sh, cache, pages, _ints(page_src, pages, "page_src"), _ints(page_dst, pages, "page_dst"), slots,
                              _ints(slot_src, slots, "slot_src"), _ints(slot_dst, slots, "slot_dst"), _stream(stream)), "moe_kv_copy")


def moe_beam_workspace_bytes(requests: int, beams: int, vocab: int, n_out: int) -> int:
    return int(load().moe_beam_workspace_bytes(requests, beams, vocab, n_out))


def moe_beam_select(logits, scores, parent, token, score, lse=None, done=None, done_out=None, end_token=-1, ws=None,
                    stream=None):
    """The best continuations of each request's beams (include/moe.h): logits [requests * beams][vocab] f32 or bf16 (rows
    possibly apart), scores [requests][beams] f32; parent, token (int32) and score (f32) [requests][n_out]; lse
    [requests][beams] f32, done [requests][beams] and done_out [requests][n_out] (bool or uint8), each or None."""
    torch = _torch or _bind_torch()
    if scores.dim() != 2 or parent.dim() != 2:
        raise ValueError("scores must be [requests][beams] and parent [requests][n_out]")
    (requests, beams), n_out, f32 = scores.shape, parent.shape[1], torch.float32
    if logits.dim() != 2 or logits.shape[0] != requests * beams or logits.dtype not in (f32, torch.bfloat16) or not logits.is_cuda:
        raise ValueError("logits must be a float32 or bfloat16 [requests * beams][vocab] GPU tensor")
    vocab, stride = logits.shape[1], logits.stride()
    if requests and vocab > 1 and stride[1] != 1:
        raise ValueError("a row's logits must be contiguous")
    for t, shape, dtypes, what in ((scores, (requests, beams), (f32,), "scores"), (parent, (requests, n_out), (torch.int32,), "parent"),
                                   (token, (requests, n_out), (torch.int32,), "token"), (score, (requests, n_out), (f32,), "score"),
                                   (lse, (requests, beams), (f32,), "lse"),
                                   (done, (requests, beams), (torch.bool, torch.uint8), "done"),
                                   (done_out, (requests, n_out), (torch.bool, torch.uint8), "done_out")):
        if t is not None and (t.shape != shape or t.dtype not in dtypes):
            raise ValueError(f"{what} must be {dtypes[0]} {list(shape)}")
    _check(load().moe_beam_select(requests, beams, vocab, n_out, logits.data_ptr(), MOE_SRC_F32 if logits.dtype is f32 else MOE_SRC_BF16,
                                  stride[0] if logits.shape[0] > 1 else vocab, _ptr(scores), _ptr(done), end_token, _ptr(parent),
                                  _ptr(token), _ptr(score), _ptr(done_out), _ptr(lse), _ptr(ws), ws.numel() if ws is not None else 0,
                                  _stream(stream)), "moe_beam_select")


def moe_linear_q4_workspace_bytes(T: int, N: int, K: int) -> int:
    return int(load().moe_linear_q4_workspace_bytes(T, N, K))


def moe_linear_q4(x, q, scales, out, residual=None, ws=None, stream=None):
    """out = x W^T (+ residual) for a few tokens, W packed int4 with group scales (include/moe.h): x [T][K] bf16 (rows
    possibly apart), q uint8 [N][K/2], scales f32 or bf16 [N][K/group], out [T][N] bf16 or f32."""
    torch = _torch or _bind_torch()
    (T, K), N, f32, bf16 = x.shape, q.shape[0], torch.float32, torch.bfloat16
    stride, groups = x.stride(), scales.shape[1]
    if x.dtype is not bf16 or not x.is_cuda or (stride[1] != 1 and T and K > 1):
        raise ValueError("x must be a bfloat16 GPU tensor with contiguous rows")
    if q.shape != (N, K // 2) or q.dtype not in (torch.uint8, torch.int8):
        raise ValueError("q must be [N][K/2] bytes")
    if scales.shape != (N, groups) or scales.dtype not in (f32, bf16) or groups == 0 or K % groups:
        raise ValueError("scales must be [N][K/group] float32 or bfloat16, group dividing K")
    if out.shape != (T, N) or out.dtype not in (f32, bf16):
        raise ValueError("out must be [T][N] float32 or bfloat16")
    if residual is not None and (residual.shape != (T, N) or residual.dtype is not bf16):
        raise ValueError("residual must be a bfloat16 [T][N] tensor")
    _check(load().moe_linear_q4(T, N, K, K // groups, x.data_ptr(), stride[0] if T > 1 else K, _ptr(q), _ptr(scales),
                                MOE_SRC_F32 if scales.dtype is f32 else MOE_SRC_BF16, _ptr(residual), _ptr(out),
                                MOE_OUT_F32 if out.dtype is f32 else 0, _ptr(ws), ws.numel() if ws is not None else 0,
                                _stream(stream)), "moe_linear_q4")


class KvPages:
    """One layer's key/value cache on the device, in the layout of include/moe.h, and its handle for the calls."""

    def __init__(self, n_pages, kv_heads, head_dim, page_tokens=64, kv_bits=8, n_slots=0, device="cuda"):
        import torch
        dt = torch.int8 if kv_bits == 8 else torch.bfloat16
        shape_k, shape_v = (kv_heads, page_tokens, head_dim), (kv_heads, head_dim, page_tokens)
        self.k = torch.empty((n_pages, *shape_k), dtype=dt, device=device)
        self.v = torch.empty((n_pages, *shape_v), dtype=dt, device=device)
        self.k_scale = self.v_scale = self.k_tail = self.v_tail = None
        if kv_bits == 8:
            self.k_scale = torch.empty((n_pages, kv_heads), dtype=torch.float32, device=device)
            self.v_scale = torch.empty((n_pages, kv_heads), dtype=torch.float32, device=device)
            self.k_tail = torch.empty((n_slots, 2, *shape_k), dtype=torch.bfloat16, device=device)
            self.v_tail = torch.empty((n_slots, 2, *shape_v), dtype=torch.bfloat16, device=device)
        self.handle = kv_cache(self.k, self.v, self.k_scale, self.v_scale, self.k_tail, self.v_tail)
        self.sizes = dict(kv_heads=kv_heads, head_dim=head_dim, kv_bits=kv_bits, page_tokens=page_tokens,
                          n_pages=n_pages, n_slots=n_slots)

    def shape(self, n_seq, rows, max_rows, max_len, q_heads, max_pages, **kw) -> MoeKvShape:
        return kv_shape(n_seq=n_seq, rows=rows, max_rows=max_rows, max_len=max_len, q_heads=q_heads,
                        max_pages=max_pages, **self.sizes, **kw)


def qmat(q, qs, q_stride_bytes: int = 0, qs_stride_floats: int = 0, q_offset: int = 0, qs_offset: int = 0) -> MoeQMat:
    """A matrix family inside device tensors q (bytes) and qs (f32), at byte / float offsets."""
    return MoeQMat(_ptr(q) + q_offset, _ptr(qs) + 4 * qs_offset, q_stride_bytes, qs_stride_floats)


class MoeLayer:
    """One layer's weights on the device, in the container layout:
    experts_q [E, 3*I*H/2] u8 (gate|up|down per expert), experts_qs [E, 2I+H] f32,
    shared_q / shared_qs likewise for the shared expert, router_w [E,H], router_bias [E]."""

    def __init__(self, cfg, arrays: dict, device="cuda"):
        import torch
        self.cfg = cfg
        dev = torch.device(device)

        def up(a):
            return None if a is None else torch.from_numpy(a).to(dev)

        self.router_w = up(arrays["router_w"])
        self.router_bias = up(arrays["router_bias"])
        self.experts_q = up(arrays["experts_q"])
        self.experts_qs = up(arrays["experts_qs"])
        self.shared_q = up(arrays.get("shared_q"))
        self.shared_qs = up(arrays.get("shared_qs"))
        self.expert_bits = up(arrays.get("expert_bits"))
        H, I, Ish = cfg.H, cfg.I, cfg.I_sh
        mat = I * H // 2
        blk, sblk = 3 * mat, 2 * I + H
        w = MoeWeights()
        w.router_w = _ptr(self.router_w)
        w.router_bias = _ptr(self.router_bias)
        w.gate = qmat(self.experts_q, self.experts_qs, blk, sblk, 0, 0)
        w.up = qmat(self.experts_q, self.experts_qs, blk, sblk, mat, I)
        w.down = qmat(self.experts_q, self.experts_qs, blk, sblk, 2 * mat, 2 * I)
        if cfg.shared_bits:
            smat = Ish * H // 2 if cfg.shared_bits == 4 else Ish * H
            w.sh_gate = qmat(self.shared_q, self.shared_qs, 0, 0, 0, 0)
            w.sh_up = qmat(self.shared_q, self.shared_qs, 0, 0, smat, Ish)
            w.sh_down = qmat(self.shared_q, self.shared_qs, 0, 0, 2 * smat, 2 * Ish)
        if self.expert_bits is not None:
            w.expert_bits = _ptr(self.expert_bits)
        self.weights = w

    def workspace(self, T: int, flags: int = 0):
        import torch
        n = moe_workspace_bytes(shape_of(self.cfg, T, flags), MOE_WS_LAYER)
        return torch.empty(n, dtype=torch.uint8, device=self.router_w.device)

    def forward(self, hidden, out, ws, flags: int = 0, stream=None):
        moe_layer_forward(shape_of(self.cfg, hidden.shape[0], flags), self.weights, hidden, out, ws, stream)
        return out

    def forward_chain(self, hidden, out, ws, flags: int = 0, nxt: Optional["MoeLayer"] = None, next_ws=None,
                      stream=None):
        """moe_layer_forward_chain: this layer, and the router logits of `nxt`
        (if given) from `out` into next_ws.  Pass MOE_LOGITS_GIVEN in flags
        when the previous layer's chained call wrote this one's logits."""
        T = hidden.shape[0]
        moe_layer_forward_chain(shape_of(self.cfg, T, flags), self.weights, hidden, out, ws,
                                shape_of(nxt.cfg, T) if nxt is not None else None,
                                nxt.weights if nxt is not None else None, next_ws, stream)
        return out
