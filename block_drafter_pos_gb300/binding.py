"""Thin ctypes binding of the C ABI in include/dflash2.h (same names, argument
marshalling only).  Tensors are torch CUDA tensors; their data pointers and the
current CUDA stream are passed straight through.  Every computation happens in
the CUDA library; there is no CPU path.  If the library has not been built, or
no GPU is present when a call needs one, the binding raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Dict, Optional

from .builder import LIB

MAX_LAYERS = 8
OK, E_INVAL, E_NONFINITE, E_CUDA, E_UNSUPPORTED, E_NO_PAGES = 0, 1, 2, 3, 4, 5
WEIGHTS_BF16, WEIGHTS_Q8G64 = 0, 1


class Dflash2Error(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: status {status} ({_status_string(status)})")
        self.status = status


class Config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "hidden", "n_layers", "n_q_heads", "n_kv_heads", "head_dim", "ffn", "vocab", "n_taps", "block",
        "top_k", "rank", "window", "conv_taps", "conv_group", "mask_token_id", "weight_format")] + [
        ("rope_theta", ctypes.c_double), ("rms_eps", ctypes.c_float)]


class Matrix(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("bias", ctypes.c_void_p)]


_LAYER_MATS = ("q", "k", "v", "o", "gate", "up", "down", "attn_delta", "mlp_delta")


class LayerWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("input_norm", "post_norm", "q_norm", "k_norm", "attn_base",
                                                 "mlp_base")] + [(n, Matrix) for n in _LAYER_MATS]


class StepArgs(ctypes.Structure):
    """dflash2_step_args: the device buffers of one draft + select + verify step."""
    _fields_ = [("n_req", ctypes.c_int32)] + [(n, ctypes.c_void_p) for n in (
        "anchor_ids", "ctx_len", "n_new", "taps", "k_cache", "v_cache", "cand_ids", "cand_logits", "gate",
        "temperature", "seed", "philox_offset", "path", "q_rows", "status", "target_logits", "n_accepted",
        "emitted", "n_emitted", "width")]


class PagedConfig(ctypes.Structure):
    """dflash2_paged_config: the geometry of one target layer's paged cache."""
    _fields_ = [(n, ctypes.c_int32) for n in ("n_q_heads", "n_kv_heads", "head_dim", "page_size", "kv_format",
                                               "max_requests")]


class PagedCache(ctypes.Structure):
    """dflash2_paged_cache: one layer's pools and the call's page table."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale", "page_table")] + [
        (n, ctypes.c_int64) for n in ("page_stride", "token_stride", "head_stride", "scale_page_stride",
                                       "scale_token_stride", "scale_head_stride", "table_stride")] + [
        ("n_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32)]


class Rows(ctypes.Structure):
    """dflash2_rows: [tokens][heads][head_dim] rows."""
    _fields_ = [("p", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("type", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class PagedAttentionArgs(ctypes.Structure):
    """dflash2_paged_attention_args."""
    _fields_ = [(n, ctypes.c_int32) for n in ("n_req", "n_tokens", "max_new", "max_len", "causal", "window")] + [
        ("scale", ctypes.c_float), ("reserved", ctypes.c_int32), ("token_begin", ctypes.c_void_p),
        ("kv_len", ctypes.c_void_p), ("q", Rows), ("out", Rows), ("tree_mask", ctypes.c_void_p),
        ("lse", ctypes.c_void_p), ("status", ctypes.c_void_p)]


class SampleArgs(ctypes.Structure):
    """dflash2_sample_args."""
    _fields_ = [(n, ctypes.c_int32) for n in ("n_rows", "vocab", "logits_type", "reserved")] + [
        ("logits", ctypes.c_void_p), ("row_stride", ctypes.c_int64)] + [
        (n, ctypes.c_void_p) for n in ("temperature", "top_k", "top_p", "min_p", "uniform", "token", "prob",
                                        "kept")] + [("kept_stride", ctypes.c_int64), ("status", ctypes.c_void_p)]


class Weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("embed", "lm_head", "hidden_norm", "final_norm")] + [
        (n, Matrix) for n in ("fc", "sel_proj", "cb_a", "cb_b")] + [("layers", LayerWeights * MAX_LAYERS)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libdflash2.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB):
            raise RuntimeError(f"libdflash2.so is not built ({LIB}); run block_drafter_pos_gb300.build()")
        L = ctypes.CDLL(LIB)
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        L.dflash2_create.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(Weights), i32, i32, ctypes.POINTER(vp)]
        L.dflash2_destroy.argtypes = [vp]
        L.dflash2_draft_block.argtypes = [vp, i32] + [vp] * 12
        L.dflash2_select.argtypes = [vp, i32] + [vp] * 13
        L.dflash2_verify.argtypes = [vp, i32] + [vp] * 14
        L.dflash2_advance.argtypes = [vp, i32] + [vp] * 7
        L.dflash2_block_width.argtypes = [vp, i32, vp, vp, i32, i32, vp, vp]
        L.dflash2_set_select_mode.argtypes = [vp, i32]
        L.dflash2_head_topk.argtypes = [vp, i32] + [vp] * 5
        L.dflash2_head_topk.restype = i32
        L.dflash2_head_topk_noalloc.argtypes = [vp, i32, i32, i32] + [vp] * 5
        L.dflash2_head_topk_noalloc.restype = i32
        L.dflash2_launch_count.argtypes = [vp]
        L.dflash2_launch_count.restype = i64
        L.dflash2_set_lmhead_events.argtypes = [vp, vp, vp]
        L.dflash2_lmhead_bytes.argtypes = [vp, i32]
        L.dflash2_lmhead_bytes.restype = i64
        L.dflash2_tree_build.argtypes = [vp, i32, i32] + [vp] * 12
        L.dflash2_tree_build.restype = i32
        L.dflash2_tree_verify.argtypes = [vp, i32, i32] + [vp] * 9
        L.dflash2_tree_verify.restype = i32
        L.dflash2_set_projection_events.argtypes = [vp, vp, i32]
        L.dflash2_set_projection_events.restype = i32
        L.dflash2_projection_launches.argtypes = [vp]
        L.dflash2_projection_launches.restype = i32
        L.dflash2_projection_bytes.argtypes = [vp]
        L.dflash2_projection_bytes.restype = i64
        L.dflash2_debug_set_pipeline_error.argtypes = [vp, vp]
        L.dflash2_debug_set_pipeline_error.restype = i32
        L.dflash2_debug_noalloc_inject_error.argtypes = [i32]
        L.dflash2_debug_noalloc_inject_error.restype = i32
        L.dflash2_step.argtypes = [vp, ctypes.POINTER(StepArgs), vp]
        L.dflash2_step.restype = i32
        L.dflash2_step_graphs_clear.argtypes = [vp]
        L.dflash2_step_graphs_clear.restype = i32
        L.dflash2_paged_create.argtypes = [ctypes.POINTER(PagedConfig), ctypes.POINTER(vp)]
        L.dflash2_paged_destroy.argtypes = [vp]
        for f in ("dflash2_paged_write", "dflash2_paged_read"):
            getattr(L, f).argtypes = [vp, ctypes.POINTER(PagedCache), i32, i32, vp, vp, ctypes.POINTER(Rows),
                                      ctypes.POINTER(Rows), vp, vp]
        L.dflash2_paged_attention.argtypes = [vp, ctypes.POINTER(PagedCache), ctypes.POINTER(PagedAttentionArgs), vp]
        L.dflash2_sample.argtypes = [ctypes.POINTER(SampleArgs), vp]
        for f in ("dflash2_paged_create", "dflash2_paged_destroy", "dflash2_paged_write", "dflash2_paged_read",
                  "dflash2_paged_attention", "dflash2_sample"):
            getattr(L, f).restype = i32
        L.dflash2_status_string.argtypes = [i32]
        L.dflash2_status_string.restype = ctypes.c_char_p
        for f in ("dflash2_create", "dflash2_destroy", "dflash2_draft_block", "dflash2_select", "dflash2_verify",
                  "dflash2_advance", "dflash2_set_select_mode",
                  "dflash2_set_lmhead_events"):
            getattr(L, f).restype = i32
        _lib = L
    return _lib


def _status_string(s: int) -> str:
    try:
        return lib().dflash2_status_string(s).decode()
    except Exception:  # noqa: BLE001 - message only
        return "?"


def _check(s: int, what: str):
    if s != OK:
        raise Dflash2Error(s, what)


def _p(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


# ----------------------------------------------------------------------------- C entry points

def dflash2_create(cfg: Config, weights: Weights, max_requests: int, kv_capacity: int) -> int:
    h = ctypes.c_void_p()
    _check(lib().dflash2_create(ctypes.byref(cfg), ctypes.byref(weights), max_requests, kv_capacity, ctypes.byref(h)),
           "dflash2_create")
    return h.value


def dflash2_destroy(h: int):
    _check(lib().dflash2_destroy(h), "dflash2_destroy")


def dflash2_draft_block(h, n_req, anchor_ids, ctx_len, n_new, taps, k_cache, v_cache, cand_ids, cand_logits, gate,
                        logits_out=None, width=None, stream=None):
    _check(lib().dflash2_draft_block(h, n_req, _p(anchor_ids), _p(ctx_len), _p(n_new), _p(taps), _p(k_cache),
                                     _p(v_cache), _p(cand_ids), _p(cand_logits), _p(gate), _p(logits_out),
                                     _p(width), _stream(stream)), "dflash2_draft_block")


def dflash2_select(h, n_req, anchor_ids, cand_ids, cand_logits, gate, temperature, seed, philox_offset, path, q_rows,
                   scores_out, status, width=None, stream=None):
    _check(lib().dflash2_select(h, n_req, _p(anchor_ids), _p(cand_ids), _p(cand_logits), _p(gate), _p(temperature),
                                _p(seed), _p(philox_offset), _p(path), _p(q_rows), _p(scores_out), _p(status),
                                _p(width), _stream(stream)), "dflash2_select")


def dflash2_verify(h, n_req, target_logits, path, cand_ids, q_rows, temperature, seed, philox_offset, n_accepted,
                   emitted, n_emitted, probs_out, status, width=None, stream=None):
    _check(lib().dflash2_verify(h, n_req, _p(target_logits), _p(path), _p(cand_ids), _p(q_rows), _p(temperature),
                                _p(seed), _p(philox_offset), _p(n_accepted), _p(emitted), _p(n_emitted),
                                _p(probs_out), _p(status), _p(width), _stream(stream)), "dflash2_verify")


def dflash2_tree_build(h, n_req, budget, anchor_ids, cand_ids, cand_logits, gate, node_token, node_parent, node_depth,
                       node_score, n_nodes, scores_out, status, stream=None):
    _check(lib().dflash2_tree_build(h, n_req, budget, _p(anchor_ids), _p(cand_ids), _p(cand_logits), _p(gate),
                                    _p(node_token), _p(node_parent), _p(node_depth), _p(node_score), _p(n_nodes),
                                    _p(scores_out), _p(status), _stream(stream)), "dflash2_tree_build")


def dflash2_tree_verify(h, n_req, budget, target_logits, node_token, node_parent, n_nodes, n_accepted, emitted,
                        n_emitted, status, stream=None):
    _check(lib().dflash2_tree_verify(h, n_req, budget, _p(target_logits), _p(node_token), _p(node_parent),
                                     _p(n_nodes), _p(n_accepted), _p(emitted), _p(n_emitted), _p(status),
                                     _stream(stream)), "dflash2_tree_verify")


def dflash2_step(h, n_req, anchor_ids, ctx_len, n_new, taps, k_cache, v_cache, cand_ids, cand_logits, gate,
                 temperature, seed, philox_offset, path, q_rows, status, target_logits, n_accepted, emitted,
                 n_emitted, width=None, stream=None):
    """One draft + select + verify step, replayed from the handle's CUDA graph of this
    argument set after its first call (dflash2.h, dflash2_step)."""
    a = StepArgs(n_req, _p(anchor_ids), _p(ctx_len), _p(n_new), _p(taps), _p(k_cache), _p(v_cache), _p(cand_ids),
                 _p(cand_logits), _p(gate), _p(temperature), _p(seed), _p(philox_offset), _p(path), _p(q_rows),
                 _p(status), _p(target_logits), _p(n_accepted), _p(emitted), _p(n_emitted), _p(width))
    _check(lib().dflash2_step(h, ctypes.byref(a), _stream(stream)), "dflash2_step")


def dflash2_step_graphs_clear(h):
    _check(lib().dflash2_step_graphs_clear(h), "dflash2_step_graphs_clear")


def dflash2_set_select_mode(h, mode: int):
    _check(lib().dflash2_set_select_mode(h, mode), "dflash2_set_select_mode")


def dflash2_advance(h, n_req, emitted, n_emitted, anchor_ids, ctx_len, n_new, philox_offset, stream=None):
    _check(lib().dflash2_advance(h, n_req, _p(emitted), _p(n_emitted), _p(anchor_ids), _p(ctx_len), _p(n_new),
                                 _p(philox_offset), _stream(stream)), "dflash2_advance")


def dflash2_block_width(h, n_req, ctx_len, n_new, ctx_threshold: int, narrow_width: int, width, stream=None):
    _check(lib().dflash2_block_width(h, n_req, _p(ctx_len), _p(n_new), ctx_threshold, narrow_width, _p(width),
                                     _stream(stream)), "dflash2_block_width")


def dflash2_head_topk(h, n_rows, hidden, cand_ids, cand_logits, logits_out=None, stream=None):
    _check(lib().dflash2_head_topk(h, n_rows, _p(hidden), _p(cand_ids), _p(cand_logits), _p(logits_out),
                                   _stream(stream)), "dflash2_head_topk")


def dflash2_head_topk_noalloc(lm_head, vocab, hidden_dim, n_rows, hidden, cand_ids, cand_logits, logits_out=None,
                              stream=None):
    """LM head + top-16 that allocates nothing: for callers that cannot call
    cudaMalloc (its scratch is a fixed device array inside the library)."""
    _check(lib().dflash2_head_topk_noalloc(_p(lm_head), vocab, hidden_dim, n_rows, _p(hidden), _p(cand_ids),
                                           _p(cand_logits), _p(logits_out), _stream(stream)),
           "dflash2_head_topk_noalloc")


def dflash2_debug_set_pipeline_error(h, stream=None):
    _check(lib().dflash2_debug_set_pipeline_error(h, _stream(stream)), "dflash2_debug_set_pipeline_error")


def dflash2_debug_noalloc_inject_error(on: bool):
    _check(lib().dflash2_debug_noalloc_inject_error(1 if on else 0), "dflash2_debug_noalloc_inject_error")


def dflash2_launch_count(h) -> int:
    return int(lib().dflash2_launch_count(h))


def dflash2_set_lmhead_events(h, start, stop):
    _check(lib().dflash2_set_lmhead_events(h, start.cuda_event if start is not None else None,
                                           stop.cuda_event if stop is not None else None),
           "dflash2_set_lmhead_events")


def dflash2_set_projection_events(h, events):
    """events: a flat list of torch.cuda.Event (start, stop, start, stop, ...), already
    created on the device (recorded once), or None.  The ctypes array is kept on the
    binding while set."""
    global _proj_events_keep
    if events is None:
        _proj_events_keep = None
        _check(lib().dflash2_set_projection_events(h, None, 0), "dflash2_set_projection_events")
        return
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    _proj_events_keep = arr
    _check(lib().dflash2_set_projection_events(h, ctypes.cast(arr, ctypes.c_void_p), len(events) // 2),
           "dflash2_set_projection_events")


_proj_events_keep = None


def dflash2_projection_launches(h) -> int:
    return int(lib().dflash2_projection_launches(h))


def dflash2_projection_bytes(h) -> int:
    return int(lib().dflash2_projection_bytes(h))


def dflash2_lmhead_bytes(h, n_req) -> int:
    return int(lib().dflash2_lmhead_bytes(h, n_req))


# ----------------------------------------------------------------------------- the target's side of a step

KV_BF16, KV_F16, KV_INT8, KV_E4M3 = 0, 1, 2, 3
T_BF16, T_F16, T_F32 = 0, 1, 2
_KV_NAMES = {"bf16": KV_BF16, "fp16": KV_F16, "int8": KV_INT8, "e4m3": KV_E4M3}
_paged_cfg: Dict[int, tuple] = {}      # geometry of each live handle, for the checks below
# The structures' bytes (checked against the header by the layout test): a packed bytes object is a
# fraction of a ctypes structure's cost, and a call's host side is all that a single token's pass waits for.
_PACK_CACHE = struct.Struct("@5P7q2i")
_PACK_ROWS = struct.Struct("@P2q2i")
_PACK_ATTN = struct.Struct("@6ifi2P" + "P2q2i" * 2 + "3P")
_PACK_SAMPLE = struct.Struct("@4iPq8PqP")
_fast = None


def _calls():
    """(torch's types, the entry points with plain pointer arguments, the current stream's handle)."""
    global _fast
    if _fast is None:
        import torch
        L = lib()
        c, vp, i32 = ctypes.c_char_p, ctypes.c_void_p, ctypes.c_int32
        fn = lambda name, *args: ctypes.CFUNCTYPE(i32, *args)((name, L))  # noqa: E731
        move = (vp, c, i32, i32, vp, vp, c, c, vp, vp)
        _fast = (torch, {torch.bfloat16: T_BF16, torch.float16: T_F16, torch.float32: T_F32},
                 {torch.bfloat16: KV_BF16, torch.float16: KV_F16, torch.int8: KV_INT8, torch.float8_e4m3fn: KV_E4M3},
                 fn("dflash2_paged_write", *move), fn("dflash2_paged_read", *move),
                 fn("dflash2_paged_attention", vp, c, c, vp), fn("dflash2_sample", c, vp))
    return _fast


def _raw_stream(what, torch, stream, dev: int) -> Optional[int]:
    """The stream's handle; a launch goes to the current device, which has to be the tensors'."""
    current = torch._C._cuda_getDevice()
    if current != dev or (stream is not None and stream.device_index != dev):
        raise _inval(what, f"the tensors are on device {dev}, which is not the current one or the stream's")
    return torch._C._cuda_getCurrentRawStream(current) if stream is None else stream.cuda_stream


def _inval(what: str, why: str):
    return Dflash2Error(E_INVAL, f"{what}: {why}")


def _vector(what, name, t, dtype, n, dev):
    """Address of a contiguous tensor of n elements on CUDA device dev, or 0 for None."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous() or t.get_device() != dev:
        raise _inval(what, f"{name} must be a contiguous tensor of {n} {dtype} on CUDA device {dev}")
    return t.data_ptr()


def _rows(what, name, t, types, heads, dim, dev):
    """The fields of dflash2_rows."""
    ty = types.get(t.dtype)
    if ty is None or t.dim() != 3 or t.get_device() != dev:
        raise _inval(what, f"{name} must be a bf16, fp16 or fp32 tensor [tokens, {heads}, {dim}] on CUDA device {dev}")
    sh, st = t.shape, t.stride()
    if sh[1] != heads or sh[2] != dim or st[2] != 1:
        raise _inval(what, f"{name} must be [tokens, {heads}, {dim}] with contiguous channels")
    return t.data_ptr(), st[0], st[1], ty, 0


def make_paged_config(n_q_heads: int, n_kv_heads: int, head_dim: int, page_size: int, kv_format: str,
                      max_requests: int) -> PagedConfig:
    """kv_format: "bf16", "fp16", "int8" or "e4m3"."""
    return PagedConfig(n_q_heads, n_kv_heads, head_dim, page_size, _KV_NAMES[kv_format], max_requests)


class PagedPool:
    """The cache structure of one layer (paged_cache makes it); it keeps the tensors alive."""
    __slots__ = ("raw", "geometry", "n_req", "device", "_keep")


def paged_cache(k, v, page_table, k_scale=None, v_scale=None) -> PagedPool:
    """The cache structure of pools k, v [pages, page_size, n_kv_heads, head_dim] (any order of
    the first three dimensions, the same for both), scales [pages, page_size, n_kv_heads]
    (8-bit pools) and page_table int32 [requests, pages of a request]."""
    what = "paged_cache"
    f = _calls()
    ty, sh, st, dev = k.dtype, k.shape, k.stride(), k.get_device()
    fmt = f[2].get(ty)
    if fmt is None or len(sh) != 4 or v.dtype is not ty:
        raise _inval(what, "k and v must be pools of one type [pages, page_size, heads, head_dim]")
    if sh != v.shape or st != v.stride() or st[3] != 1 or dev < 0 or v.get_device() != dev:
        raise _inval(what, "k and v must be tensors of one shape and layout on one CUDA device, with contiguous channels")
    torch, rows, along = f[0], page_table.shape, page_table.stride()
    if page_table.dtype is not torch.int32 or len(rows) != 2 or page_table.get_device() != dev or along[1] != 1:
        raise _inval(what, "page_table must be an int32 tensor [requests, pages] on the pools' device, with contiguous rows")
    c = PagedPool()
    c.device = dev
    c.n_req, max_pages = rows
    ks = vs = 0
    ss = (0, 0, 0)
    if fmt >= KV_INT8:
        if k_scale is None or v_scale is None or k_scale.dtype is not torch.float32 or v_scale.dtype is not torch.float32 or \
                k_scale.shape != sh[:3] or v_scale.shape != sh[:3] or k_scale.get_device() != dev or v_scale.get_device() != dev:
            raise _inval(what, "8-bit pools need float32 scales [pages, page_size, heads] on the pools' device")
        ss = k_scale.stride()
        if ss != v_scale.stride():
            raise _inval(what, "the scales must have one layout")
        ks, vs = k_scale.data_ptr(), v_scale.data_ptr()
    c.raw = _PACK_CACHE.pack(k.data_ptr(), v.data_ptr(), ks, vs, page_table.data_ptr(), st[0], st[1], st[2], *ss,
                             along[0] if c.n_req > 1 else max_pages, sh[0], max_pages)
    c.geometry = (fmt, sh[1], sh[2], sh[3])
    c._keep = (k, v, page_table, k_scale, v_scale)
    return c


def dflash2_paged_create(cfg: PagedConfig) -> int:
    h = ctypes.c_void_p()
    _check(lib().dflash2_paged_create(ctypes.byref(cfg), ctypes.byref(h)), "dflash2_paged_create")
    _paged_cfg[h.value] = ((cfg.kv_format, cfg.page_size, cfg.n_kv_heads, cfg.head_dim), cfg.n_q_heads,
                           _calls()[0]._C._cuda_getDevice())
    return h.value


def dflash2_paged_destroy(h: int):
    if h not in _paged_cfg:
        raise _inval("dflash2_paged_destroy", "not a paged handle")
    _check(lib().dflash2_paged_destroy(h), "dflash2_paged_destroy")
    _paged_cfg.pop(h, None)


def _paged_check(what, torch, h, cache, token_begin, kv_len, status):
    """The handle's geometry and device against the cache's; returns (geometry, query heads, requests, three addresses)."""
    g = _paged_cfg.get(h)
    if g is None:
        raise _inval(what, "not a paged handle")
    if cache.geometry != g[0]:
        raise _inval(what, "the pools are not of the handle's format, page size or heads")
    dev = cache.device
    if dev != g[2]:
        raise _inval(what, f"the pools are on device {dev}, the handle on {g[2]}")
    n = kv_len.numel()
    if n > cache.n_req:
        raise _inval(what, "the page table has fewer rows than there are requests")
    i32 = torch.int32
    return g[0], g[1], n, _vector(what, "token_begin", token_begin, i32, n + 1, dev), \
        _vector(what, "kv_len", kv_len, i32, n, dev), _vector(what, "status", status, i32, n, dev)


def _paged_move(what, which, h, cache, k, v, token_begin, kv_len, status, stream):
    f = _calls()
    g, _, n, begin, length, st = _paged_check(what, f[0], h, cache, token_begin, kv_len, status)
    if k.shape != v.shape or k.dtype is not v.dtype:
        raise _inval(what, "k and v must have one shape and type")
    dev = cache.device
    rk, rv = _rows(what, "k", k, f[1], g[2], g[3], dev), _rows(what, "v", v, f[1], g[2], g[3], dev)
    s = f[which](h, cache.raw, n, k.shape[0], begin, length, _PACK_ROWS.pack(*rk), _PACK_ROWS.pack(*rv), st,
                 _raw_stream(what, f[0], stream, dev))
    if s:
        _check(s, what)


def dflash2_paged_write(h, cache, k, v, token_begin, kv_len, status=None, stream=None):
    """Writes the new tokens' keys and values [tokens, n_kv_heads, head_dim] into their positions."""
    _paged_move("dflash2_paged_write", 3, h, cache, k, v, token_begin, kv_len, status, stream)


def dflash2_paged_read(h, cache, k, v, token_begin, kv_len, status=None, stream=None):
    """Reads the same positions back into k and v."""
    _paged_move("dflash2_paged_read", 4, h, cache, k, v, token_begin, kv_len, status, stream)


def dflash2_paged_attention(h, cache, q, out, token_begin, kv_len, max_new, max_len, scale, causal=True, window=0,
                            tree_mask=None, lse=None, status=None, stream=None):
    """Attention of the new tokens q [tokens, n_q_heads, head_dim] over their requests' caches, into out.
    tree_mask: int64 [tokens] (the bits of a uint64)."""
    what = "dflash2_paged_attention"
    f = _calls()
    torch = f[0]
    g, hq, n, begin, length, st = _paged_check(what, torch, h, cache, token_begin, kv_len, status)
    dev = cache.device
    rq, ro = _rows(what, "q", q, f[1], hq, g[3], dev), _rows(what, "out", out, f[1], hq, g[3], dev)
    tokens = q.shape[0]
    if out.shape[0] != tokens:
        raise _inval(what, "q and out must have the same rows")
    a = _PACK_ATTN.pack(n, tokens, max_new, max_len, 1 if causal else 0, window, scale, 0, begin, length, *rq, *ro,
                        _vector(what, "tree_mask", tree_mask, torch.int64, tokens, dev),
                        _vector(what, "lse", lse, torch.float32, tokens * hq, dev), st)
    s = f[5](h, cache.raw, a, _raw_stream(what, torch, stream, dev))
    if s:
        _check(s, what)


def dflash2_sample(logits, temperature, top_k, top_p, min_p, uniform, token, prob=None, kept=None, status=None,
                   stream=None):
    """Truncated sampling of the rows of logits [rows, vocab]; top_k, top_p and min_p may be None."""
    what = "dflash2_sample"
    f = _calls()
    torch = f[0]
    ty = f[1].get(logits.dtype)
    dev = logits.get_device()
    if ty is None or logits.dim() != 2 or logits.stride(1) != 1 or dev < 0:
        raise _inval(what, "logits must be a bf16, fp16 or fp32 CUDA tensor [rows, vocab] with contiguous rows")
    n, v = logits.shape
    i32, f32 = torch.int32, torch.float32
    if kept is not None and (kept.dtype is not f32 or kept.shape != logits.shape or kept.stride(1) != 1 or kept.get_device() != dev):
        raise _inval(what, "kept must be a float32 tensor of the logits' shape and device with contiguous rows")
    a = _PACK_SAMPLE.pack(n, v, ty, 0, logits.data_ptr(), logits.stride(0),
                          _vector(what, "temperature", temperature, f32, n, dev), _vector(what, "top_k", top_k, i32, n, dev),
                          _vector(what, "top_p", top_p, f32, n, dev), _vector(what, "min_p", min_p, f32, n, dev),
                          _vector(what, "uniform", uniform, f32, n, dev), _vector(what, "token", token, i32, n, dev),
                          _vector(what, "prob", prob, f32, n, dev), 0 if kept is None else kept.data_ptr(),
                          0 if kept is None else kept.stride(0), _vector(what, "status", status, i32, n, dev))
    s = f[6](a, _raw_stream(what, torch, stream, dev))
    if s:
        _check(s, what)


# ----------------------------------------------------------------------------- convenience

def make_config(geom, weight_format: str) -> Config:
    c = Config()
    for n in ("hidden", "n_layers", "n_q_heads", "n_kv_heads", "head_dim", "ffn", "vocab", "n_taps", "block",
              "top_k", "rank", "window", "conv_taps", "conv_group"):
        setattr(c, n, getattr(geom, n))
    c.mask_token_id = geom.mask_id
    c.weight_format = WEIGHTS_BF16 if weight_format == "bf16" else WEIGHTS_Q8G64
    c.rope_theta = geom.rope_theta
    c.rms_eps = geom.rms_eps
    return c


def upload_weights(W: Dict[str, object], device="cuda"):
    """Copies a weight dict (numpy, layout of workloads.gen) to the device.  Returns
    (dict of torch tensors keeping them alive, ctypes Weights)."""
    import numpy as np
    import torch

    keep = {}

    def dev(name, arr):
        a = np.ascontiguousarray(arr)
        if a.dtype == np.uint16:
            a = a.view(np.int16)
        t = torch.from_numpy(a).to(device)
        keep[name] = t
        return t.data_ptr()

    def mat(name, m):
        x = Matrix()
        if m["kind"] == "bf16":
            x.w = dev(name, m["w"])
        else:
            x.w = dev(name + ".codes", m["codes"])
            x.scale = dev(name + ".scale", m["scale"])
            x.bias = dev(name + ".bias", m["bias"])
        return x

    w = Weights()
    for n in ("embed", "lm_head", "hidden_norm", "final_norm"):
        setattr(w, n, dev(n, W[n]))
    for n in ("fc", "sel_proj", "cb_a", "cb_b"):
        setattr(w, n, mat(n, W[n]))
    l = 0
    while f"l{l}.q" in W:
        L = w.layers[l]
        p = f"l{l}."
        for n in ("input_norm", "post_norm", "q_norm", "k_norm", "attn_base", "mlp_base"):
            setattr(L, n, dev(p + n, W[p + n]))
        for n in _LAYER_MATS:
            setattr(L, n, mat(p + n, W[p + n]))
        l += 1
    return keep, w


class Drafter:
    """Owns a handle and the device weights of one synthetic drafter."""

    def __init__(self, geom, weight_format: str, W: Dict[str, object], max_requests: int, kv_capacity: int):
        self.geom = geom
        self.cfg = make_config(geom, weight_format)
        self._keep, self._w = upload_weights(W)
        self.max_requests = max_requests
        self.kv_capacity = kv_capacity
        self.handle = dflash2_create(self.cfg, self._w, max_requests, kv_capacity)

    def close(self):
        if self.handle:
            dflash2_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:  # noqa: BLE001
            pass
