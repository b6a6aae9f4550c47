"""The calls for many samples of one prompt without a GPU: refusals, structure layouts, the rotation's plan, the binding's
checks, and the oracle's pins."""
import ctypes
import math
import os
import shutil
import subprocess
import types

import numpy as np
import pytest
import torch

import block_drafter_pos_gb300 as bd
from block_drafter_pos_gb300 import serving as sv
from oracle import serving as os_
from test_target_calls import Stub
from test_target_host import BAD_CACHE, BAD_ROWS, FakeHandle, P, _attn, _cache, _rows

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
b = bd.binding


# ----------------------------------------------------------------------------- the rotation's plan

def _config(**kw):
    c = sv.RopeConfig(64, 0, sv.ROPE_PLAIN, 0, 1e4, 1.0, 0.0, 0.0, 0.0, None)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


NAN, INF = float("nan"), float("inf")
BAD_PLANS = [(dict(rot_dim=0), "E_INVAL"), (dict(rot_dim=-16), "E_INVAL"), (dict(rot_dim=24), "E_UNSUPPORTED"),
             (dict(rot_dim=272), "E_UNSUPPORTED"), (dict(interleaved=2), "E_INVAL"), (dict(scaling=4), "E_INVAL"),
             (dict(scaling=-1), "E_INVAL"), (dict(theta=1.0), "E_INVAL"), (dict(theta=NAN), "E_INVAL"), (dict(theta=INF), "E_INVAL"),
             (dict(amplitude=-1.0), "E_INVAL"), (dict(amplitude=NAN), "E_INVAL"), (dict(amplitude=1e39), "E_INVAL"),
             (dict(scaling=1, factor=0.0), "E_INVAL"), (dict(scaling=1, factor=-2.0), "E_INVAL"), (dict(scaling=1, factor=1e-9), "E_INVAL"),
             (dict(scaling=2, factor=0.5, original_len=9), "E_INVAL"), (dict(scaling=2, factor=2.0), "E_INVAL"),
             (dict(scaling=2, factor=2.0, original_len=9, beta_fast=NAN), "E_INVAL"),
             (dict(scaling=2, factor=2.0, original_len=9, beta_slow=-1.0), "E_INVAL"), (dict(scaling=3), "E_INVAL")]


@pytest.mark.parametrize("kw,want", BAD_PLANS)
def test_plan_refuses_bad_settings(kw, want):
    out = sv.Rotation()
    assert bd.lib().dflash2_rope_plan(ctypes.byref(_config(**kw)), ctypes.byref(out)) == getattr(b, want)
    assert bd.lib().dflash2_rope_plan(None, ctypes.byref(out)) == b.E_INVAL
    assert bd.lib().dflash2_rope_plan(ctypes.byref(_config()), None) == b.E_INVAL


@pytest.mark.parametrize("bad", [NAN, INF, 2.0 ** 21])
def test_plan_refuses_rates_out_of_bounds(bad):
    with pytest.raises(bd.Dflash2Error):
        bd.make_rope(16, scaling="table", table=[0.1] * 7 + [bad])
    with pytest.raises(bd.Dflash2Error):
        bd.make_rope(16, scaling="table", table=[0.1] * 7)
    with pytest.raises(bd.Dflash2Error):
        bd.make_rope(16, scaling="other")


@pytest.mark.parametrize("kw", [dict(), dict(theta=1e4), dict(scaling="linear", factor=8.0),
                                dict(scaling="yarn", factor=4.0, original_len=32768),
                                dict(scaling="yarn", factor=16.0, original_len=4096, beta_fast=24.0, beta_slow=2.0, theta=1e4),
                                dict(scaling="yarn", factor=2.0, original_len=3)])
@pytest.mark.parametrize("rot", [16, 96, 256])
def test_plan_holds_the_rates_as_turns(kw, rot):
    """The plan's turns times 2 pi are the formula's rates: FP64 on both sides, a few roundings of 2^-53 and one of 2^-65 of
    a turn (the low word is cut, not rounded: 2^-64)."""
    p = sv.Rotation.from_buffer_copy(bd.make_rope(rot, **kw).raw)
    rates, amplitude = os_.rope_rates(rot, **dict(dict(theta=1e7), **kw))
    got = np.array([int(x) for x in p.turns[:rot // 2]], dtype=np.float64) * 2.0 ** -64 * 2 * math.pi
    assert np.all(np.abs(got - rates) <= 2.0 ** -49 * rates + 2.0 ** -60)
    assert abs(p.amplitude - amplitude) <= 2.0 ** -24 * amplitude and not any(p.turns[rot // 2:])
    assert p.rot_dim == rot


def test_plan_takes_a_table():
    rates = [0.5, -0.25, 0.0, 7.0, 100.0, -2.0 ** 20, 1e-9, -1e-30]
    p = sv.Rotation.from_buffer_copy(bd.make_rope(16, scaling="table", table=rates, amplitude=0.75, interleaved=True).raw)
    for x, f in zip(p.turns, rates):
        turn = f / (2 * math.pi)
        d = abs(int(x) * 2.0 ** -64 - (turn - math.floor(turn)))
        assert min(d, 1 - d) <= 2.0 ** -50 * abs(turn) + 2.0 ** -52
    assert p.amplitude == 0.75 and p.interleaved == 1


# ----------------------------------------------------------------------------- refusals

def _plan(rot=64):
    return bytes(bd.make_rope(rot).raw)


def _rotation(**kw):
    r = sv.Rotation.from_buffer_copy(_plan())
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def _raw(r):
    return ctypes.cast(ctypes.byref(r), ctypes.c_char_p) if r is not None else None


def _call_rope(plan=None, n=4, dim=128, heads=2, x=None, out=None, k_heads=0, k=None, k_out=None, positions=P):
    f = bd.lib().dflash2_rope
    vp = ctypes.c_void_p
    f.argtypes = [vp, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, vp, vp, ctypes.c_int32, vp, vp, vp, ctypes.c_int32, vp]
    f.restype = ctypes.c_int32
    ref = lambda r: ctypes.addressof(r) if r is not None else None  # noqa: E731
    return f(ref(plan), n, dim, heads, ref(x), ref(out), k_heads, ref(k), ref(k_out), positions, 0, None)


def test_rope_refuses_bad_arguments():
    ok, far = _rotation(), 1 << 30
    x, y = _rows(), _rows(p=far)
    assert _call_rope(None, x=x, out=y) == b.E_INVAL
    for kw in (dict(rot_dim=0), dict(rot_dim=24), dict(rot_dim=512), dict(interleaved=5), dict(amplitude=NAN)):
        assert _call_rope(_rotation(**kw), x=x, out=y) == b.E_INVAL, kw
    for kw in (dict(n=-1), dict(dim=0), dict(heads=-1), dict(k_heads=-1), dict(positions=None)):
        assert _call_rope(ok, **{**dict(x=x, out=y), **kw}) == b.E_INVAL, kw
    for kw in (dict(dim=100), dict(dim=2048), dict(dim=56), dict(heads=1025), dict(heads=600, k_heads=500), dict(n=2 ** 31 - 15)):
        assert _call_rope(ok, **{**dict(x=x, out=y, k=x, k_out=y), **kw}) == b.E_UNSUPPORTED, kw
    for kw in BAD_ROWS:
        assert _call_rope(ok, x=_rows(**kw), out=y) == b.E_INVAL, kw
        assert _call_rope(ok, x=x, out=_rows(**{**dict(p=far), **kw})) == b.E_INVAL, kw
        assert _call_rope(ok, x=x, out=y, k_heads=1, k=_rows(**kw), k_out=y) == b.E_INVAL, kw
    assert _call_rope(ok, x=None, out=y) == b.E_INVAL and _call_rope(ok, x=x, out=None) == b.E_INVAL
    assert _call_rope(ok, x=x, out=y, k_heads=1) == b.E_INVAL
    assert _call_rope(ok, x=x, out=_rows(p=far, type=b.T_F16)) == b.E_INVAL
    assert _call_rope(ok, x=x, out=y, k_heads=1, k=_rows(type=b.T_F16), k_out=_rows(p=far, type=b.T_F16)) == b.E_INVAL
    # overlapping rows that are not the same rows: 4 tokens of 2 heads of 128, strides 256 and 128
    for at in (16, 256 * 2, (3 * 256 + 128 + 127) * 2 // 16 * 16):
        assert _call_rope(ok, x=x, out=_rows(p=P + at)) == b.E_INVAL, at
        assert _call_rope(ok, x=_rows(p=P + at), out=x) == b.E_INVAL, at
    assert _call_rope(ok, x=x, out=_rows(token_stride=512)) == b.E_INVAL
    assert _call_rope(ok, x=_rows(token_stride=-256), out=_rows(p=P - 3 * 512)) == b.E_INVAL
    # nothing to do is no error
    assert _call_rope(ok, n=0) == b.OK and _call_rope(ok, heads=0) == b.OK


def _call_write(h, plan, cache, n_req=1, n=4, begin=P, kv=P, q=None, q_out=None, k=None, v=None):
    f = bd.lib().dflash2_paged_rope_write
    vp, i32 = ctypes.c_void_p, ctypes.c_int32
    f.argtypes, f.restype = [vp, vp, vp, i32, i32] + [vp] * 9, i32
    ref = lambda r: ctypes.addressof(r) if r is not None else None  # noqa: E731
    return f(h, ref(plan), ref(cache), n_req, n, begin, kv, None, ref(q), ref(q_out), ref(k), ref(v), None, None)


def test_rope_write_refuses_bad_arguments():
    h, c, r, plan, far = FakeHandle(), _cache(), _rows(), _rotation(), 1 << 30
    q = _rows(token_stride=1024)
    assert _call_write(None, plan, c, k=r, v=r) == b.E_INVAL
    assert _call_write(h.p, None, c, k=r, v=r) == b.E_INVAL
    assert _call_write(h.p, plan, None, k=r, v=r) == b.E_INVAL
    assert _call_write(h.p, _rotation(rot_dim=24), c, k=r, v=r) == b.E_INVAL
    assert _call_write(h.p, _rotation(rot_dim=144), c, k=r, v=r) == b.E_UNSUPPORTED       # above head_dim
    assert _call_write(h.p, plan, c, n_req=5, k=r, v=r) == b.E_UNSUPPORTED
    assert _call_write(h.p, plan, c, n=2 ** 31 - 15, k=r, v=r) == b.E_UNSUPPORTED
    for kw in (dict(n=-1), dict(n_req=-1), dict(begin=None), dict(kv=None), dict(k=None), dict(v=None), dict(v=_rows(type=b.T_F16)),
               dict(q=q), dict(q=q, q_out=_rows(p=far, token_stride=1024, type=b.T_F16)),
               dict(q=_rows(token_stride=1024, type=b.T_F16), q_out=_rows(p=far, token_stride=1024, type=b.T_F16)),
               dict(q=q, q_out=_rows(p=P + 2048, token_stride=1024))):
        assert _call_write(h.p, plan, c, **{**dict(k=r, v=r), **kw}) == b.E_INVAL, kw
    for kw in BAD_CACHE:
        assert _call_write(h.p, plan, _cache(**kw), k=r, v=r) == b.E_INVAL, kw
    for kw in BAD_ROWS:
        assert _call_write(h.p, plan, c, k=_rows(**kw), v=r) == b.E_INVAL, kw
        assert _call_write(h.p, plan, c, k=r, v=r, q=_rows(**kw), q_out=_rows(p=far)) == b.E_INVAL, kw
    assert _call_write(h.p, plan, c, n=0, k=r, v=r) == b.OK and _call_write(h.p, plan, _cache(page_table=None), n_req=0, k=r, v=r) == b.OK


def _pool(**kw):
    d = dict(ref=P, table=P, stride=8, n_pages=100, n_rows=4, max_pages=8, page=16)
    d.update(kw)
    return sv._PACK_POOL.pack(*(d[k] or 0 for k in ("ref", "table", "stride", "n_pages", "n_rows", "max_pages", "page")))


BAD_POOLS = [(dict(ref=None), "E_INVAL"), (dict(table=None), "E_INVAL"), (dict(stride=7), "E_INVAL"), (dict(n_pages=0), "E_INVAL"),
             (dict(n_rows=-1), "E_INVAL"), (dict(max_pages=0), "E_INVAL"), (dict(page=0), "E_INVAL"),
             (dict(n_pages=(1 << 22) + 1), "E_UNSUPPORTED"), (dict(n_rows=1025), "E_UNSUPPORTED")]


def test_pages_calls_refuse_bad_arguments():
    f = sv._calls()
    resize, fork = f["resize"], f["fork"]
    for kw, want in BAD_POOLS:
        assert resize(_pool(**kw), P, P + 64, P, None, None) == getattr(b, want), kw
        assert fork(_pool(**kw), 1, P, P, P, None, None) == getattr(b, want), kw
    assert resize(None, P, P + 64, P, None, None) == b.E_INVAL and fork(None, 1, P, P, P, None, None) == b.E_INVAL
    for args in ((None, P, P), (P, None, P), (P, P + 64, None), (P, P, P)):
        assert resize(_pool(), *args, None, None) == b.E_INVAL, args
    assert resize(_pool(n_rows=0, table=None), None, None, None, None, None) == b.OK
    for args in ((-1, P, P, P), (1, None, P, P), (1, P, None, P), (1, P, P, None)):
        assert fork(_pool(), *args, None, None) == b.E_INVAL, args
    assert fork(_pool(n_rows=0, table=None), 1, P, P, P, None, None) == b.E_INVAL
    assert fork(_pool(), 1025, P, P, P, None, None) == b.E_UNSUPPORTED
    assert fork(_pool(), 0, None, None, None, None, None) == b.OK


def _two(**kw):
    """Two layers' structures, the second with a change."""
    return bytes(_cache()) + bytes(_cache(**kw))


def test_copy_and_keep_refuse_bad_arguments():
    f, h = sv._calls(), FakeHandle()
    copy, keep = f["copy"], f["keep"]
    good = (1, P, P, P, 4, 4, P, None)          # requests, begin, kv_len, keep, stride, most, n_keep, kv_out
    assert copy(None, 2, _two(), 1, P, None, None) == b.E_INVAL and keep(None, 2, _two(), *good, None, None) == b.E_INVAL
    assert copy(h.p, 2, None, 1, P, None, None) == b.E_INVAL and keep(h.p, 2, None, *good, None, None) == b.E_INVAL
    for kw in BAD_CACHE:
        assert keep(h.p, 2, _two(**kw), *good, None, None) == b.E_INVAL, kw
        if not set(kw) & {"page_table", "table_stride", "max_pages"}:
            assert copy(h.p, 2, _two(**kw), 1, P, None, None) == b.E_INVAL, kw
    assert copy(h.p, -1, _two(), 1, P, None, None) == b.E_INVAL and copy(h.p, 2, _two(), -1, P, None, None) == b.E_INVAL
    assert copy(h.p, 2, _two(), 1, None, None, None) == b.E_INVAL and copy(h.p, 2, _two(), (1 << 20) + 1, P, None, None) == b.E_UNSUPPORTED
    assert copy(h.p, 2, _two(), 0, None, None, None) == b.OK and copy(h.p, 0, None, 1, P, None, None) == b.OK
    for i, bad in ((0, -1), (1, None), (2, None), (3, None), (5, -1), (6, None), (7, P)):
        args = good[:i] + (bad,) + good[i + 1:]
        assert keep(h.p, 2, _two(), *args, None, None) == b.E_INVAL, (i, bad)
    assert keep(h.p, 0, _two(), *good, None, None) == b.E_INVAL
    assert keep(h.p, 2, _two(), 5, *good[1:], None, None) == b.E_UNSUPPORTED                 # more than max_requests
    assert keep(h.p, 2, _two(), 2, P, P, P, 3, 4, P, None, None, None) == b.E_INVAL          # overlapping rows of keep
    assert keep(h.p, 2, _two(page_table=None), 0, None, None, None, 4, 4, None, None, None, None) == b.OK


def _shared(tokens=4, groups=1, max_group=4, max_prefix=16, begin=P, prefix=P, work=P, size=1 << 40, how=0, **kw):
    a = _attn(n_tokens=tokens, **kw)
    return bytes(a) + sv._PACK_SHARED.pack(groups, max_group, max_prefix, how, begin or 0, prefix or 0, work or 0, size)


def test_shared_attention_refuses_bad_arguments():
    f, h, c = sv._calls()["shared"], FakeHandle(), bytes(_cache())
    need = 4 * 8 * 130 * 4
    assert bd.lib().dflash2_paged_shared_bytes(h.p, 4) == need and bd.lib().dflash2_paged_shared_bytes(None, 4) == 0
    assert bd.lib().dflash2_paged_shared_bytes(h.p, -1) == 0
    assert f(None, c, _shared(), None) == b.E_INVAL and f(h.p, None, _shared(), None) == b.E_INVAL and f(h.p, c, None, None) == b.E_INVAL
    for kw in BAD_CACHE:
        assert f(h.p, bytes(_cache(**kw)), _shared(), None) == b.E_INVAL, kw
    for kw in BAD_ROWS + [dict(type=b.T_F32)]:
        assert f(h.p, c, _shared(q=_rows(**kw)), None) == b.E_INVAL, kw
        assert f(h.p, c, _shared(out=_rows(**kw)), None) == b.E_INVAL, kw
    for kw in (dict(window=1), dict(groups=-1), dict(groups=0), dict(max_group=-1), dict(max_prefix=-1), dict(begin=None),
               dict(prefix=None), dict(how=-1), dict(how=3), dict(work=None), dict(work=P + 16), dict(size=need - 1), dict(scale=NAN), dict(max_len=-1)):
        assert f(h.p, c, _shared(**kw), None) == b.E_INVAL, kw
    assert f(h.p, c, _shared(groups=1025), None) == b.E_UNSUPPORTED
    assert f(h.p, c, _shared(n_req=5), None) == b.E_UNSUPPORTED
    assert f(h.p, c, _shared(tokens=1 << 30, max_group=1 << 30), None) == b.E_UNSUPPORTED
    for kw in (dict(tokens=0), dict(max_new=0), dict(n_req=0, groups=0, work=None)):
        assert f(h.p, c, _shared(**kw), None) == b.OK, kw


# ----------------------------------------------------------------------------- layouts, the binding

def test_binding_structures_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    exe = str(tmp_path / "layout")
    subprocess.run([cc, "-std=c99", "-I", os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "abi_layout_serving.c"),
                    "-o", exe], check=True)
    got = dict(line.split() for line in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines())
    at = b._PACK_ATTN.size
    want = {"dflash2_rope_config": ctypes.sizeof(sv.RopeConfig), "dflash2_rope_config.theta": sv.RopeConfig.theta.offset,
            "dflash2_rope_config.amplitude": sv.RopeConfig.amplitude.offset, "dflash2_rope_config.table": sv.RopeConfig.table.offset,
            "dflash2_rotation": ctypes.sizeof(sv.Rotation), "dflash2_rotation.amplitude": sv.Rotation.amplitude.offset,
            "dflash2_rotation.turns": sv.Rotation.turns.offset,
            "dflash2_page_pool": sv._PACK_POOL.size, "dflash2_page_pool.table_stride": 16, "dflash2_page_pool.n_pages": 24,
            "dflash2_page_pool.page_size": 36,
            "dflash2_paged_shared_args": at + sv._PACK_SHARED.size, "dflash2_paged_shared_args.n_groups": at,
            "dflash2_paged_shared_args.group_begin": at + 16, "dflash2_paged_shared_args.workspace": at + 32,
            "dflash2_paged_shared_args.workspace_bytes": at + 40}
    assert {k: int(v) for k, v in got.items()} == want


@pytest.fixture
def calls(monkeypatch):
    """The entry points replaced by ones that note the call; the current device is the first entry."""
    made, current = [], [0]
    real, mine = b._calls(), sv._calls()
    note = lambda *a: made.append(a) or b.OK  # noqa: E731
    fake = types.SimpleNamespace(int32=torch.int32, int64=torch.int64, float32=torch.float32, uint8=torch.uint8, _C=types.SimpleNamespace(
        _cuda_getDevice=lambda: current[0], _cuda_getCurrentRawStream=lambda d: 77 + d))
    monkeypatch.setattr(b, "_fast", (fake,) + real[1:])
    monkeypatch.setattr(sv, "_fast", {k: v if k in ("types", "plan") else note for k, v in mine.items()})
    monkeypatch.setitem(b._paged_cfg, 4096, ((b.KV_INT8, 16, 2, 128), 8, 0))
    return made, current


BF, I32 = torch.bfloat16, torch.int32
TENSORS = dict(x=(BF, 6, 8, 128), out=(BF, 6, 8, 128), k=(BF, 6, 2, 128), k_out=(BF, 6, 2, 128), v=(BF, 6, 2, 128),
               positions=(I32, 6), begin=(I32, 4), kv_len=(I32, 3), new_len=(I32, 3), copies=(I32, 3, 3), status=(I32, 3), parent=(I32, 3),
               child=(I32, 3), keep=(I32, 3, 4), n_keep=(I32, 3), kv_out=(I32, 3), group_begin=(I32, 3), prefix=(I32, 2),
               work=(torch.uint8, 1 << 20), tree=(torch.int64, 6), lse=(torch.float32, 6, 8), table=(I32, 3, 4), ref=(I32, 9))


def _cache_on(dev=0):
    f32, i8 = torch.float32, torch.int8
    return bd.paged_cache(Stub(dev, i8, 9, 16, 2, 128), Stub(dev, i8, 9, 16, 2, 128), Stub(dev, I32, 3, 4), Stub(dev, f32, 9, 16, 2),
                          Stub(dev, f32, 9, 16, 2))


def _each_call(dev=0, stream=None, cache=None, change=None, **other):
    """Every call, with the names of what it takes; `other`: tensors on another device, `change`: tensors of another shape or type."""
    t = {k: Stub(other.get(k, dev), *(change or {}).get(k, v)) for k, v in TENSORS.items()}
    c = cache or _cache_on(dev)
    rope, s = bd.make_rope(64), dict(stream=stream)
    pool = lambda: bd.page_pool(t["table"], t["ref"], 16)  # noqa: E731
    yield "x out positions k k_out", lambda: bd.dflash2_rope(rope, t["x"], t["out"], t["positions"], k=t["k"], k_out=t["k_out"], **s)
    yield "x out k v begin kv_len positions status", lambda: bd.dflash2_paged_rope_write(
        4096, rope, c, t["x"], t["out"], t["k"], t["v"], t["begin"], t["kv_len"], t["positions"], t["status"], **s)
    yield "table ref kv_len new_len copies status", lambda: bd.dflash2_pages_resize(
        pool(), t["kv_len"], t["new_len"], t["copies"], t["status"], **s)
    yield "table ref parent child kv_len status", lambda: bd.dflash2_pages_fork(
        pool(), t["parent"], t["child"], t["kv_len"], t["status"], **s)
    yield "copies status", lambda: bd.dflash2_pages_copy(4096, [c, c], t["copies"], t["status"], **s)
    yield "begin kv_len keep n_keep kv_out status", lambda: bd.dflash2_paged_keep(
        4096, [c, c], t["begin"], t["kv_len"], t["keep"], t["n_keep"], t["kv_out"], t["status"], **s)
    yield "x out begin kv_len group_begin prefix work tree lse status", lambda: bd.dflash2_paged_attention_shared(
        4096, c, t["x"], t["out"], t["begin"], t["kv_len"], t["group_begin"], t["prefix"], t["work"], 6, 64, 6, 16, 0.1,
        tree_mask=t["tree"], lse=t["lse"], status=t["status"], **s)


def test_calls_on_one_device_go_through(calls):
    made, _ = calls
    for _, call in _each_call():
        call()
    assert len(made) == 7 and all(m[-1] == 77 for m in made)
    for _, call in _each_call(stream=types.SimpleNamespace(device_index=0, cuda_stream=5)):
        call()
    assert len(made) == 14 and all(m[-1] == 5 for m in made[7:])


@pytest.mark.parametrize("where", [1, -1])
def test_tensors_of_several_devices_are_refused(calls, where):
    made, _ = calls
    for name in TENSORS:
        for takes, call in _each_call(**{name: where}):
            if name in takes.split():
                with pytest.raises(bd.Dflash2Error):
                    call()
            else:
                call()
    takes = [t.split() for t, _ in _each_call()]
    assert len(made) == sum(name not in t for name in TENSORS for t in takes)


def test_shapes_and_types_are_checked(calls):
    made, _ = calls
    for name, bad in dict(x=(BF, 6, 7, 120), out=(BF, 5, 8, 128), k=(BF, 5, 2, 128), k_out=(BF, 6, 3, 128), v=(torch.float16, 6, 2, 128),
                          positions=(torch.int64, 6), begin=(I32, 3), new_len=(I32, 4), copies=(I32, 2, 3),
                          status=(I32, 2), parent=(I32, 2), child=(I32, 4), keep=(I32, 2, 4), n_keep=(I32, 4), kv_out=(torch.int64, 3),
                          group_begin=(I32, 2), tree=(torch.int64, 5), lse=(torch.float32, 6, 7), ref=(torch.int64, 9)).items():
        for takes, call in _each_call(change={name: bad}):
            if name in takes.split():
                with pytest.raises(bd.Dflash2Error):
                    call()
                    pytest.fail(f"{name}: {takes}")
    assert not [m for m in made if m is None]


def test_another_device_than_the_current_one_is_refused(calls):
    made, current = calls
    other = types.SimpleNamespace(device_index=1, cuda_stream=5)
    for stream in (None, other):
        current[0] = 1 if stream is None else 0
        for _, call in _each_call(stream=stream):
            with pytest.raises(bd.Dflash2Error, match="current"):
                call()
    assert not made


def test_unknown_handles_are_refused(calls):
    c = _cache_on()
    with pytest.raises(bd.Dflash2Error):
        bd.dflash2_pages_copy(4097, [c], Stub(0, I32, 3, 3))
    with pytest.raises(bd.Dflash2Error):
        bd.dflash2_paged_shared_bytes(None, 4)
    with pytest.raises(bd.Dflash2Error, match="how"):
        t = {k: Stub(0, *v) for k, v in TENSORS.items()}
        bd.dflash2_paged_attention_shared(4096, c, t["x"], t["out"], t["begin"], t["kv_len"], t["group_begin"], t["prefix"], t["work"], 6,
                                          64, 6, 16, 0.1, how="other")


# ----------------------------------------------------------------------------- the oracle's pins

def test_oracle_rotation_is_a_product_of_complex_numbers():
    g = np.random.default_rng(0)
    x, pos = g.standard_normal((5, 3, 24)), np.array([0, 1, 7, -3, 1000])
    rates, _ = os_.rope_rates(16, 1e4)
    for inter in (False, True):
        y, _ = os_.rope(x, pos, rates, 1.5, inter)
        i = np.arange(8)
        a, c = (2 * i, 2 * i + 1) if inter else (i, i + 8)
        z = (x[..., a] + 1j * x[..., c]) * np.exp(1j * pos[:, None] * rates)[:, None] * 1.5
        assert np.allclose(y[..., a], z.real, atol=1e-12) and np.allclose(y[..., c], z.imag, atol=1e-12)
        assert np.array_equal(y[..., 16:], x[..., 16:]) and np.array_equal(y[0, :, 16:], x[0, :, 16:])
        back, _ = os_.rope(y, pos, rates, 1 / 1.5, inter, inverse=True)
        assert np.allclose(back, x, atol=1e-12)


def test_oracle_pages_by_hand():
    """Pages of 4 positions: a prompt of 6, two samples of it, each one's first token, and all given back."""
    table = [[-1] * 4 for _ in range(3)]
    ref, kv = [0] * 8, [0, 0, 0]
    assert os_.pages_resize(table, ref, kv, [6, 0, 0], 4) == ([(-1, -1, 0)] * 3, [0, 0, 0])
    assert table[0] == [0, 1, -1, -1] and ref == [1, 1] + [0] * 6 and kv == [6, 0, 0]
    assert os_.pages_fork(table, ref, kv, [0, 0], [1, 2], 4) == [0, 0]
    assert table[1] == table[2] == [0, 1, -1, -1] and ref[:2] == [3, 3] and kv == [6, 6, 6]
    # the samples grow, the prompt does not: both copy
    t, f, k = [list(r) for r in table], list(ref), list(kv)
    assert os_.pages_resize(t, f, k, [6, 7, 9], 4)[0] == [(-1, -1, 0), (1, 2, 2), (1, 3, 2)]
    assert t == [[0, 1, -1, -1], [0, 2, -1, -1], [0, 3, 4, -1]] and f == [3, 1, 1, 1, 1, 0, 0, 0]
    # all three grow: the first keeps the page
    assert os_.pages_resize(table, ref, kv, [7, 7, 7], 4)[0] == [(-1, -1, 0), (1, 2, 2), (1, 3, 2)]
    assert ref == [3, 1, 1, 1, 0, 0, 0, 0]
    # the second wants more than there is, so the third gets nothing either; the first needs nothing
    assert os_.pages_resize(table, ref, kv, [8, 16, 9], 4)[1] == [0, 0, 0]
    assert os_.pages_resize(table, ref, kv, [8, 16, 16], 4)[1] == [0, 0, 0] and ref == [3, 1, 1, 1, 1, 1, 1, 1][:8]
    assert os_.pages_resize(table, ref, kv, [9, 16, 16], 4)[1] == [5, 0, 0] and kv == [8, 16, 16]
    assert os_.pages_resize(table, ref, kv, [0, 0, 0], 4)[1] == [0, 0, 0] and not any(ref) and table == [[-1] * 4] * 3
    assert os_.pages_fork(table, ref, kv, [0, 0, 1, 2], [1, 1, 2, 0], 4) == [1, 1, 1, 1]


def test_a_wait_that_gives_up_spoils_its_run():
    """Every role of the prefix's kernel marks its CTA, and partials that never come are NaN; the joining kernel flags a run's groups."""
    csrc = os.path.join(ROOT, "block_drafter_pos_gb300", "csrc")
    text, sched = (open(os.path.join(csrc, n)).read() for n in ("paged_prefix.cu", "paged_sched.cuh"))
    assert text.count("a.desc[8 * c + 6] = 1;") == 4 and text.count("a.desc[8 * c + 6] = 0;") == 1
    assert text.index("make_float2(NAN, NAN)") < text.index("tcgen05.alloc") and "paged_flag<kShared>(a, r, 3)" in open(
        os.path.join(csrc, "paged_attention.cu")).read()
    assert "for (int x = __ldg(a.g.begin + r); x < __ldg(a.g.begin + r + 1); ++x) a.rq.status[x] = what;" in sched
