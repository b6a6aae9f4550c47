"""Binding of the calls for many samples of one prompt: rotary positions, the pages of a pool, and attention
over shared prefixes (include/dflash2.h; same names, argument marshalling and checks only, as in binding.py)."""
from __future__ import annotations

import ctypes
import struct
from typing import Optional, Sequence

from . import binding as _b
from .binding import _check, _inval, _raw_stream, _rows, _vector

ROPE_PLAIN, ROPE_LINEAR, ROPE_YARN, ROPE_TABLE = 0, 1, 2, 3
ROPE_MAX_DIM = 256
_SCALING = {"none": ROPE_PLAIN, "linear": ROPE_LINEAR, "yarn": ROPE_YARN, "table": ROPE_TABLE}
_HOW = {"auto": 0, "together": 1, "apart": 2}
_PACK_POOL = struct.Struct("@2Pq4i")
_PACK_SHARED = struct.Struct("@4i3Pq")      # behind the attention's arguments


class RopeConfig(ctypes.Structure):
    """dflash2_rope_config."""
    _fields_ = [(n, ctypes.c_int32) for n in ("rot_dim", "interleaved", "scaling", "original_len")] + [
        (n, ctypes.c_double) for n in ("theta", "factor", "beta_fast", "beta_slow", "amplitude")] + [
        ("table", ctypes.POINTER(ctypes.c_double))]


class Rotation(ctypes.Structure):
    """dflash2_rotation: the plan of a rotation (make_rope makes it)."""
    _fields_ = [("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("amplitude", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("turns", ctypes.c_uint64 * (ROPE_MAX_DIM // 2))]


_fast = None


def _calls():
    """The entry points with plain pointer arguments, and the types of rows."""
    global _fast
    if _fast is None:
        L = _b.lib()
        c, vp, i32, i64 = ctypes.c_char_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        fn = lambda name, *args: ctypes.CFUNCTYPE(i32, *args)((name, L))  # noqa: E731
        _fast = {
            "types": _b._calls()[1],
            "plan": fn("dflash2_rope_plan", vp, vp),
            "rope": fn("dflash2_rope", c, i32, i32, i32, c, c, i32, c, c, vp, i32, vp),
            "write": fn("dflash2_paged_rope_write", vp, c, c, i32, i32, vp, vp, vp, c, c, c, c, vp, vp),
            "resize": fn("dflash2_pages_resize", c, vp, vp, vp, vp, vp),
            "fork": fn("dflash2_pages_fork", c, i32, vp, vp, vp, vp, vp),
            "copy": fn("dflash2_pages_copy", vp, i32, c, i32, vp, vp, vp),
            "keep": fn("dflash2_paged_keep", vp, i32, c, i32, vp, vp, vp, i64, i32, vp, vp, vp, vp),
            "shared": fn("dflash2_paged_attention_shared", vp, c, c, vp),
        }
        L.dflash2_paged_shared_bytes.argtypes = [vp, i32]
        L.dflash2_paged_shared_bytes.restype = i64
    return _fast


# ----------------------------------------------------------------------------- rotary positions

class RopePlan:
    """A rotation as the calls take it (make_rope makes it): plain host data, of no device."""
    __slots__ = ("raw", "rot_dim", "interleaved", "amplitude")


def make_rope(rot_dim: int, theta: float = 1e7, interleaved: bool = False, scaling: str = "none", factor: float = 1.0,
              original_len: int = 0, beta_fast: float = 0.0, beta_slow: float = 0.0, amplitude: float = 0.0,
              table: Optional[Sequence[float]] = None) -> RopePlan:
    """scaling: "none", "linear", "yarn" or "table" (radians per position of each pair); the formulas are the header's."""
    what = "dflash2_rope_plan"
    if scaling not in _SCALING:
        raise _inval(what, f"scaling must be one of {', '.join(_SCALING)}")
    values = None
    if table is not None:
        if len(table) != rot_dim // 2:
            raise _inval(what, f"table must have {rot_dim // 2} entries")
        values = (ctypes.c_double * len(table))(*[float(x) for x in table])
    cfg = RopeConfig(rot_dim, int(interleaved), _SCALING[scaling], original_len, theta, factor, beta_fast, beta_slow, amplitude,
                     values)
    r = Rotation()
    _check(_calls()["plan"](ctypes.addressof(cfg), ctypes.addressof(r)), what)
    p = RopePlan()
    p.raw, p.rot_dim, p.interleaved, p.amplitude = bytes(r), r.rot_dim, bool(r.interleaved), r.amplitude
    return p


def _pair(what, names, x, y, types, dev):
    """Two tensors of one shape and type, as rows.  (Checked together: what a short call costs is this side of it.)"""
    ty, sx, sy = types.get(x.dtype), x.stride(), y.stride()
    if ty is None or len(sx) != 3 or x.shape != y.shape or x.dtype is not y.dtype or sx[2] != 1 or sy[2] != 1 or \
            x.get_device() != dev or y.get_device() != dev:
        raise _inval(what, f"{names[0]} and {names[1]} must be bf16, fp16 or fp32 tensors of one shape [tokens, heads, head_dim] and "
                           f"type with contiguous channels on CUDA device {dev}")
    pack = _b._PACK_ROWS.pack
    return pack(x.data_ptr(), sx[0], sx[1], ty, 0), pack(y.data_ptr(), sy[0], sy[1], ty, 0)


def dflash2_rope(rope: RopePlan, x, out, positions, k=None, k_out=None, inverse=False, stream=None):
    """Turns rows x [tokens, heads, head_dim] by positions int32 [tokens] into out (may be x), and k into k_out in the same
    launch; inverse: by the opposite angle (the gradient's way back)."""
    what = "dflash2_rope"
    f, torch = _calls(), _b._calls()[0]
    dev = x.get_device()
    if dev < 0:
        raise _inval(what, "x must be a CUDA tensor")
    rx, ry = _pair(what, ("x", "out"), x, out, f["types"], dev)
    n, heads, dim = x.shape
    rk = rk_out = None
    k_heads = 0
    if (k is None) != (k_out is None):
        raise _inval(what, "k and k_out come together")
    if k is not None:
        if k.dim() != 3 or k.shape[0] != n or k.shape[2] != dim or k.dtype is not x.dtype:
            raise _inval(what, "k must have x's tokens, head_dim and type")
        rk, rk_out = _pair(what, ("k", "k_out"), k, k_out, f["types"], dev)
        k_heads = k.shape[1]
    s = f["rope"](rope.raw, n, dim, heads, rx, ry, k_heads, rk, rk_out, _vector(what, "positions", positions, torch.int32, n, dev),
                  1 if inverse else 0, _raw_stream(what, torch, stream, dev))
    if s:
        _check(s, what)


def dflash2_paged_rope_write(h, rope: RopePlan, cache, q, q_out, k, v, token_begin, kv_len, positions=None, status=None,
                             stream=None):
    """Writes the turned keys and the values [tokens, n_kv_heads, head_dim] into their positions, and the turned queries
    [tokens, n_q_heads, head_dim] into q_out (may be q; both None: keys and values only).  positions: int32 [tokens] in
    the place of the cache's positions."""
    what = "dflash2_paged_rope_write"
    f, torch = _calls(), _b._calls()[0]
    g, hq, n, begin, length, st = _b._paged_check(what, torch, h, cache, token_begin, kv_len, status)
    dev, shape = cache.device, k.shape
    rk, rv = _pair(what, ("k", "v"), k, v, f["types"], dev)
    tokens = shape[0]
    if shape[1:] != g[2:]:
        raise _inval(what, f"k and v must have {g[2]} heads of {g[3]}")
    rq = ry = None
    if (q is None) != (q_out is None):
        raise _inval(what, "q and q_out come together")
    if q is not None:
        if q.shape != (tokens, hq, g[3]) or q.dtype is not k.dtype:
            raise _inval(what, f"q must have k's tokens and type, {hq} heads of {g[3]}")
        rq, ry = _pair(what, ("q", "q_out"), q, q_out, f["types"], dev)
    s = f["write"](h, rope.raw, cache.raw, n, tokens, begin, length,
                   _vector(what, "positions", positions, torch.int32, tokens, dev), rq, ry, rk, rv, st,
                   _raw_stream(what, torch, stream, dev))
    if s:
        _check(s, what)


# ----------------------------------------------------------------------------- the pages of a pool

class PagePool:
    """The page table and the counts of holders of a pool (page_pool makes it); it keeps the tensors alive."""
    __slots__ = ("raw", "n_rows", "device", "_keep")


def page_pool(page_table, ref, page_size: int, h: Optional[int] = None) -> PagePool:
    """page_table int32 [rows, pages of a row], ref int32 [pages] (zeros at the start): the pool's state, which the calls change.
    h: the paged handle whose caches go by the table, to have its page size and device compared."""
    what = "page_pool"
    torch = _b._calls()[0]
    if h is not None:
        g = _b._paged_cfg.get(h)
        if g is None:
            raise _inval(what, "not a paged handle")
        if g[0][1] != page_size or g[2] != page_table.get_device():
            raise _inval(what, f"the handle's pages have {g[0][1]} positions, on device {g[2]}")
    dev = page_table.get_device()
    if page_table.dtype is not torch.int32 or page_table.dim() != 2 or dev < 0 or page_table.stride(1) != 1:
        raise _inval(what, "page_table must be an int32 CUDA tensor [rows, pages], with contiguous rows")
    n, width = page_table.shape
    if n > 1 and page_table.stride(0) < width:
        raise _inval(what, "the page table's rows overlap")
    p = PagePool()
    p.n_rows, p.device = n, dev
    p.raw = _PACK_POOL.pack(_vector(what, "ref", ref, torch.int32, ref.numel(), dev), page_table.data_ptr(),
                            page_table.stride(0) if n > 1 else width, ref.numel(), n, width, page_size)
    p._keep = (page_table, ref)
    return p


def dflash2_pages_resize(pool: PagePool, kv_len, new_len, copies, status=None, stream=None):
    """Every row from kv_len to new_len positions (int32 [rows]; kv_len is brought up to date): pages taken, given back, and
    noted for copying in copies int32 [3, rows]."""
    what = "dflash2_pages_resize"
    f, torch = _calls(), _b._calls()[0]
    n, dev, i32 = pool.n_rows, pool.device, torch.int32
    s = f["resize"](pool.raw, _vector(what, "kv_len", kv_len, i32, n, dev), _vector(what, "new_len", new_len, i32, n, dev),
                    _vector(what, "copies", copies, i32, 3 * n, dev), _vector(what, "status", status, i32, n, dev),
                    _raw_stream(what, torch, stream, dev))
    if s:
        _check(s, what)


def dflash2_pages_fork(pool: PagePool, parent, child, kv_len, status=None, stream=None):
    """Row child[i] becomes another holder of row parent[i]'s pages, with its length (parent, child int32 [pairs])."""
    what = "dflash2_pages_fork"
    f, torch = _calls(), _b._calls()[0]
    n, dev, i32 = parent.numel(), pool.device, torch.int32
    s = f["fork"](pool.raw, n, _vector(what, "parent", parent, i32, n, dev), _vector(what, "child", child, i32, n, dev),
                  _vector(what, "kv_len", kv_len, i32, pool.n_rows, dev), _vector(what, "status", status, i32, n, dev),
                  _raw_stream(what, torch, stream, dev))
    if s:
        _check(s, what)


def _layers(what, h, caches):
    """(geometry, device, the structures of the layers' pools one after the other)."""
    g = _b._paged_cfg.get(h)
    if g is None:
        raise _inval(what, "not a paged handle")
    geometry, dev = g[0], g[2]
    for c in caches:
        if c.geometry != geometry or c.device != dev:
            raise _inval(what, "the pools are not of the handle's format, page size or heads" if c.device == dev else
                         f"the pools are on device {c.device}, the handle on {dev}")
    return geometry, dev, b"".join([c.raw for c in caches])


def dflash2_pages_copy(h, caches, copies, status=None, stream=None):
    """The copies (int32 [3, n]) that dflash2_pages_resize noted, in each layer's pools."""
    what = "dflash2_pages_copy"
    f, torch = _calls(), _b._calls()[0]
    _, dev, raw = _layers(what, h, caches)
    if copies.dim() != 2 or copies.shape[0] != 3:
        raise _inval(what, "copies must be an int32 tensor [3, n]")
    n = copies.shape[1]
    s = f["copy"](h, len(caches), raw, n, _vector(what, "copies", copies, torch.int32, 3 * n, dev),
                  _vector(what, "status", status, torch.int32, n, dev), _raw_stream(what, torch, stream, dev))
    if s:
        _check(s, what)


def dflash2_paged_keep(h, caches, token_begin, kv_len, keep, n_keep, kv_out=None, status=None, stream=None):
    """Moves new tokens keep[r, : n_keep[r]] (int32, ascending) of each request to its first new places, in each layer's
    pools; kv_out: the lengths after that."""
    what = "dflash2_paged_keep"
    f, torch = _calls(), _b._calls()[0]
    _, dev, raw = _layers(what, h, caches)
    n, i32 = kv_len.numel(), torch.int32
    if any(n > c.n_req for c in caches):
        raise _inval(what, "a page table has fewer rows than there are requests")
    if keep.dtype is not i32 or keep.dim() != 2 or keep.shape[0] != n or keep.get_device() != dev or (keep.shape[1] > 1 and keep.stride(1) != 1):
        raise _inval(what, f"keep must be an int32 tensor [{n}, most kept] on CUDA device {dev}, with contiguous rows")
    s = f["keep"](h, len(caches), raw, n, _vector(what, "token_begin", token_begin, i32, n + 1, dev),
                  _vector(what, "kv_len", kv_len, i32, n, dev), keep.data_ptr(), keep.stride(0) if n > 1 else keep.shape[1],
                  keep.shape[1], _vector(what, "n_keep", n_keep, i32, n, dev), _vector(what, "kv_out", kv_out, i32, n, dev),
                  _vector(what, "status", status, i32, n, dev), _raw_stream(what, torch, stream, dev))
    if s:
        _check(s, what)


# ----------------------------------------------------------------------------- attention over shared prefixes

def dflash2_paged_shared_bytes(h, n_tokens: int) -> int:
    """Bytes of the workspace of dflash2_paged_attention_shared with n_tokens rows."""
    if h not in _b._paged_cfg:
        raise _inval("dflash2_paged_shared_bytes", "not a paged handle")
    _calls()
    return int(_b.lib().dflash2_paged_shared_bytes(h, n_tokens))


def dflash2_paged_attention_shared(h, cache, q, out, token_begin, kv_len, group_begin, prefix_len, workspace, max_new, max_len,
                                   max_group, max_prefix, scale, causal=True, tree_mask=None, lse=None, status=None, how="auto",
                                   stream=None):
    """dflash2_paged_attention where requests group_begin[g] .. group_begin[g + 1] - 1 (int32 [groups + 1]) share their first
    prefix_len[g] positions (int32 [groups]), whose keys and values are read through its first request's
    row of the page table.  workspace: uint8 [dflash2_paged_shared_bytes(h, tokens)].
    how: "together", "apart" or "auto"."""
    what = "dflash2_paged_attention_shared"
    f, torch = _calls(), _b._calls()[0]
    types, i32 = f["types"], torch.int32
    g, hq, n, begin, length, st = _b._paged_check(what, torch, h, cache, token_begin, kv_len, status)
    dev = cache.device
    rq, ro = _rows(what, "q", q, types, hq, g[3], dev), _rows(what, "out", out, types, hq, g[3], dev)
    tokens, groups = q.shape[0], prefix_len.numel()
    if out.shape[0] != tokens:
        raise _inval(what, "q and out must have the same rows")
    room = workspace.numel()
    a = _b._PACK_ATTN.pack(n, tokens, max_new, max_len, 1 if causal else 0, 0, scale, 0, begin, length, *rq, *ro,
                           _vector(what, "tree_mask", tree_mask, torch.int64, tokens, dev),
                           _vector(what, "lse", lse, torch.float32, tokens * hq, dev), st)
    if how not in _HOW:
        raise _inval(what, f"how must be one of {', '.join(_HOW)}")
    a += _PACK_SHARED.pack(groups, max_group, max_prefix, _HOW[how], _vector(what, "group_begin", group_begin, i32, groups + 1, dev),
                           _vector(what, "prefix_len", prefix_len, i32, groups, dev), _vector(what, "workspace", workspace, torch.uint8, room, dev), room)
    s = f["shared"](h, cache.raw, a, _raw_stream(what, torch, stream, dev))
    if s:
        _check(s, what)
