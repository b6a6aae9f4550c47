"""The target's side of a step (paged cache, attention over it, truncated sampling) without a
GPU: refusals, structure layouts, the attention's schedule, and the oracle's pins."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import block_drafter_pos_gb300 as bd
from oracle import target as ot

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
b = bd.binding
P = 1 << 20          # a 16-byte aligned address that nothing dereferences


# ----------------------------------------------------------------------------- refusals

@pytest.mark.parametrize("kw,want", [
    (dict(head_dim=96), "E_UNSUPPORTED"),
    (dict(head_dim=256), "E_UNSUPPORTED"),
    (dict(head_dim=0), "E_INVAL"),
    (dict(n_q_heads=12), "E_UNSUPPORTED"),            # not a multiple of the KV heads
    (dict(n_q_heads=8 * 65), "E_UNSUPPORTED"),        # more than 64 query heads per KV head
    (dict(n_kv_heads=0), "E_INVAL"),
    (dict(page_size=0), "E_INVAL"),
    (dict(page_size=-16), "E_INVAL"),
    (dict(kv_format=4), "E_INVAL"),
    (dict(kv_format=-1), "E_INVAL"),
    (dict(max_requests=0), "E_INVAL"),
    (dict(max_requests=1025), "E_UNSUPPORTED"),
])
def test_create_refuses_geometry_before_any_device_call(kw, want):
    cfg = b.PagedConfig(32, 8, 128, 16, b.KV_BF16, 4)
    for k, v in kw.items():
        setattr(cfg, k, v)
    h = ctypes.c_void_p(7)
    assert bd.lib().dflash2_paged_create(ctypes.byref(cfg), ctypes.byref(h)) == getattr(b, want)
    assert not h.value
    assert bd.lib().dflash2_paged_create(None, ctypes.byref(h)) == b.E_INVAL
    assert bd.lib().dflash2_paged_destroy(None) == b.E_INVAL


class FakeHandle:
    """A handle's memory with the configuration at its start, as the checks read it: every call below is
    refused before a kernel or the scratch is touched."""

    def __init__(self, fmt=b.KV_INT8, max_requests=4):
        self.buf = (ctypes.c_char * 256)()
        cfg = b.PagedConfig(8, 2, 128, 16, fmt, max_requests)
        ctypes.memmove(self.buf, ctypes.byref(cfg), ctypes.sizeof(cfg))
        self.p = ctypes.cast(self.buf, ctypes.c_void_p)


def _cache(**kw):
    c = b.PagedCache(P, P, P, P, P, 16 * 2 * 128, 2 * 128, 128, 32, 2, 1, 64, 100, 64)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _rows(**kw):
    r = b.Rows(P, 256, 128, b.T_BF16, 0)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


BAD_CACHE = [dict(k=None), dict(v=None), dict(k=P + 8), dict(v=P + 2), dict(k_scale=None), dict(v_scale=None),
             dict(page_table=None), dict(n_pages=0), dict(max_pages=0), dict(table_stride=63), dict(page_stride=4097),
             dict(token_stride=257), dict(head_stride=120)]
BAD_ROWS = [dict(p=None), dict(p=P + 4), dict(type=3), dict(type=-1), dict(token_stride=257), dict(head_stride=4)]


@pytest.mark.parametrize("call", ["dflash2_paged_write", "dflash2_paged_read"])
def test_write_and_read_refuse_bad_arguments(call):
    f, h = getattr(bd.lib(), call), FakeHandle()
    c, r = _cache(), _rows()
    assert f(None, c, 1, 1, P, P, r, r, None, None) == b.E_INVAL
    assert f(h.p, None, 1, 1, P, P, r, r, None, None) == b.E_INVAL
    assert f(h.p, c, -1, 1, P, P, r, r, None, None) == b.E_INVAL
    assert f(h.p, c, 5, 1, P, P, r, r, None, None) == b.E_UNSUPPORTED     # more than max_requests
    assert f(h.p, c, 1, -1, P, P, r, r, None, None) == b.E_INVAL
    assert f(h.p, c, 1, 1, None, P, r, r, None, None) == b.E_INVAL
    assert f(h.p, c, 1, 1, P, None, r, r, None, None) == b.E_INVAL
    assert f(h.p, c, 1, 1, P, P, None, r, None, None) == b.E_INVAL
    assert f(h.p, c, 1, 1, P, P, r, _rows(type=b.T_F16), None, None) == b.E_INVAL
    for kw in BAD_CACHE:
        assert f(h.p, _cache(**kw), 1, 1, P, P, r, r, None, None) == b.E_INVAL, kw
    for kw in BAD_ROWS:
        assert f(h.p, c, 1, 1, P, P, _rows(**kw), r, None, None) == b.E_INVAL, kw
        assert f(h.p, c, 1, 1, P, P, r, _rows(**kw), None, None) == b.E_INVAL, kw
    # nothing to do is no error
    assert f(h.p, c, 0, 0, P, P, r, r, None, None) == b.OK
    assert f(h.p, c, 1, 0, P, P, r, r, None, None) == b.OK


def _attn(**kw):
    a = b.PagedAttentionArgs(1, 4, 4, 64, 1, 0, 0.1, 0, P, P, _rows(), _rows(), None, None, None)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_attention_refuses_bad_arguments():
    f, h, c = bd.lib().dflash2_paged_attention, FakeHandle(), _cache()
    assert f(None, c, _attn(), None) == b.E_INVAL
    assert f(h.p, c, None, None) == b.E_INVAL
    for kw in BAD_CACHE:
        assert f(h.p, _cache(**kw), _attn(), None) == b.E_INVAL, kw
    for kw in BAD_ROWS + [dict(type=b.T_F32)]:
        assert f(h.p, c, _attn(q=_rows(**kw)), None) == b.E_INVAL, kw
        assert f(h.p, c, _attn(out=_rows(**kw)), None) == b.E_INVAL, kw
    for kw in [dict(n_req=-1), dict(n_tokens=-1), dict(max_new=-1), dict(max_len=-1), dict(window=-1),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(token_begin=None), dict(kv_len=None),
               dict(q=_rows(type=b.T_F16))]:
        assert f(h.p, c, _attn(**kw), None) == b.E_INVAL, kw
    assert f(h.p, c, _attn(n_req=5), None) == b.E_UNSUPPORTED
    assert f(h.p, c, _attn(tree_mask=P, max_new=65, n_tokens=65), None) == b.E_UNSUPPORTED
    # a 16-bit cache takes queries of its own type only
    assert f(FakeHandle(b.KV_F16).p, c, _attn(), None) == b.E_INVAL
    for kw in [dict(n_tokens=0), dict(max_new=0), dict(n_req=0)]:
        assert f(h.p, c, _attn(**kw), None) == b.OK, kw


def test_sample_refuses_bad_arguments():
    f = bd.lib().dflash2_sample

    def args(**kw):
        a = b.SampleArgs(2, 100, b.T_F32, 0, P, 100, P, P, P, P, P, P, P, 4 * P, 100, P)
        for k, v in kw.items():
            setattr(a, k, v)
        return a

    assert f(None, None) == b.E_INVAL
    for kw in [dict(n_rows=-1), dict(vocab=0), dict(logits_type=3), dict(logits=None), dict(temperature=None),
               dict(uniform=None), dict(token=None), dict(row_stride=99), dict(kept_stride=99)]:
        assert f(args(**kw), None) == b.E_INVAL, kw
    # kept over the logits: the same rows only
    for kw in [dict(kept=P + 4), dict(kept=P - 400), dict(kept_stride=200), dict(logits_type=b.T_F16)]:
        assert f(args(**{"kept": P, **kw}), None) == b.E_INVAL, kw
    assert f(args(vocab=(1 << 19) + 1, row_stride=1 << 20, kept_stride=1 << 20), None) == b.E_UNSUPPORTED
    assert f(args(n_rows=0), None) == b.OK


def test_binding_refuses_wrong_tensors():
    k = torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16)
    table = torch.zeros(1, 4, dtype=torch.int32)
    for args in [(k, k, table), (k, k[:, :8], table), (k.float(), k.float(), table), (k, k.half(), table)]:
        with pytest.raises(bd.Dflash2Error):
            bd.paged_cache(*args)                       # not CUDA tensors, or not one type and shape
    with pytest.raises(bd.Dflash2Error):
        bd.dflash2_paged_write(12345, None, k, k, table, table)
    x = torch.zeros(2, 50)
    with pytest.raises(bd.Dflash2Error):
        bd.dflash2_sample(x, x, None, None, None, x, x)


def test_structures_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    exe = str(tmp_path / "layout")
    subprocess.run([cc, "-std=c99", "-I", os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "abi_layout_target.c"), "-o", exe], check=True)
    lines = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines()
    cls = {"dflash2_paged_config": b.PagedConfig, "dflash2_paged_cache": b.PagedCache, "dflash2_rows": b.Rows,
           "dflash2_paged_attention_args": b.PagedAttentionArgs, "dflash2_sample_args": b.SampleArgs}
    assert len(lines) == 21
    for packed, name in [(b._PACK_CACHE, "dflash2_paged_cache"), (b._PACK_ROWS, "dflash2_rows"),
                         (b._PACK_ATTN, "dflash2_paged_attention_args"), (b._PACK_SAMPLE, "dflash2_sample_args")]:
        assert packed.size == ctypes.sizeof(cls[name])
    for line in lines:
        name, value = line.split()
        t, _, field = name.partition(".")
        got = getattr(cls[t], field).offset if field else ctypes.sizeof(cls[t])
        assert got == int(value), name


def test_schedule_and_bounds_against_brute_force(tmp_path):
    gxx = shutil.which("g++")
    inc = "/usr/local/cuda/include"
    if gxx is None or not os.path.exists(os.path.join(inc, "cuda.h")):
        pytest.skip("g++ or the CUDA headers are missing")
    exe = str(tmp_path / "check")
    subprocess.run([gxx, "-std=c++17", "-O2", "-I", os.path.join(ROOT, "block_drafter_pos_gb300", "csrc"), "-I", inc,
                    os.path.join(ROOT, "tests", "paged_schedule_check.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout
    assert out.stdout.startswith("ok ") and int(out.stdout.split()[1]) > 10000


def test_packed_bytes_are_the_structures():
    r = b.Rows(1, 2, 3, 1, 0)
    assert bytes(b.PagedCache(*range(1, 15))) == b._PACK_CACHE.pack(*range(1, 15))
    assert bytes(r) == b._PACK_ROWS.pack(1, 2, 3, 1, 0)
    assert bytes(b.PagedAttentionArgs(1, 2, 3, 4, 5, 6, 0.5, 0, 7, 8, r, r, 9, 10, 11)) == \
        b._PACK_ATTN.pack(1, 2, 3, 4, 5, 6, 0.5, 0, 7, 8, 1, 2, 3, 1, 0, 1, 2, 3, 1, 0, 9, 10, 11)
    assert bytes(b.SampleArgs(1, 2, 0, 0, *range(4, 16))) == b._PACK_SAMPLE.pack(1, 2, 0, 0, *range(4, 16))


# ----------------------------------------------------------------------------- the oracle's pins

def test_oracle_e4m3_rounding_against_the_type():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    codes = np.unique(codes[np.isfinite(codes)])
    assert len(codes) == 253                                   # 2 * 126 values and zero
    np.testing.assert_array_equal(ot.e4m3_round(codes), codes)
    mid = (codes[1:] + codes[:-1]) / 2
    x = np.concatenate([mid, np.nextafter(mid, -1e9), np.nextafter(mid, 1e9), np.linspace(-448, 448, 9001)])
    got = ot.e4m3_round(x)
    near = np.abs(codes[None] - x[:, None]).min(1)
    np.testing.assert_allclose(np.abs(got - x), near, rtol=0, atol=0)     # always a nearest value
    t = torch.tensor(x, dtype=torch.float32)
    exact = t.double().numpy() == x                            # ties to even as the type's conversion has them
    np.testing.assert_array_equal(got[exact], t.to(torch.float8_e4m3fn).float().numpy()[exact])


@pytest.mark.parametrize("fmt,half", [("int8", 0.5), ("e4m3", 16.0)])
def test_oracle_quantise(fmt, half):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((50, 64)).astype(np.float32) * np.exp(rng.uniform(-20, 20, (50, 1))).astype(np.float32)
    x[7] = 0
    codes, scale = ot.quantise(x, fmt)
    q = ot.QMAX[fmt]
    assert np.abs(codes).max() == q and (np.abs(codes).max(-1)[np.arange(50) != 7] == q).all()
    assert scale[7] == np.float32(2.0 ** -126) and not codes[7].any()
    err = np.abs(codes * scale[:, None].astype(np.float64) - x)
    assert (err <= scale[:, None] * half * (1 + 1e-6)).all()              # at most half of the largest step
    x[3, 5], x[4, 6] = np.nan, -np.inf
    codes, scale = ot.quantise(x, fmt)
    assert not codes[3:5].any() and np.isnan(scale[3]) and np.isinf(scale[4])


def test_oracle_attention_against_dense_softmax():
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(s, generator=g, dtype=torch.float64) for s in [(6, 4, 64), (40, 2, 64), (40, 2, 64)])
    see = ot.visible(6, 40)
    np.testing.assert_array_equal(see, np.tril(np.ones((6, 40), bool), 34))
    out, lse, spread, reach = ot.paged_attention(q, k, v, 0.125, see)
    kk, vv = k.repeat_interleave(2, 1), v.repeat_interleave(2, 1)
    s = torch.einsum("nhd,mhd->hnm", q, kk) * 0.125
    s.masked_fill_(~torch.tensor(see), float("-inf"))
    np.testing.assert_allclose(out, torch.einsum("hnm,mhd->nhd", s.softmax(-1), vv), rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(lse, s.logsumexp(-1).T, rtol=1e-12)
    assert (spread >= np.abs(out) - 1e-12).all() and (reach >= s.abs().nan_to_num(0, 0, 0).amax(-1).T.numpy() - 1e-9).all()
    # windows, trees, rows that see nothing
    w = ot.visible(6, 40, True, 3)
    assert (w.sum(1) == 3).all() and w[5, 37:].all()
    t = ot.visible(3, 10, tree=[1, 3, 5])
    np.testing.assert_array_equal(t[:, 7:], [[1, 0, 0], [1, 1, 0], [1, 0, 1]])
    assert t[:, :7].all()
    out, lse, _, _ = ot.paged_attention(q[:3], k[:2], v[:2], 1.0, ot.visible(3, 2))   # positions -1, 0, 1
    assert not out[0].any() and np.isneginf(lse[0]).all() and np.array_equal(out[1], v[0].repeat_interleave(2, 0))


def test_oracle_sample_against_its_definition():
    rng = np.random.default_rng(9)
    for trial in range(200):
        v = int(rng.integers(2, 12))
        x = rng.integers(-3, 4, v).astype(np.float64)          # many equal logits
        t, k, p, m = rng.uniform(0.3, 2), int(rng.integers(0, v + 2)), rng.choice([1.0, 0.5, 0.83]), rng.choice([0.0, 0.2])
        prob = np.exp(x / t) / np.exp(x / t).sum()
        left = sorted(range(v), key=lambda i: (-x[i], i))[:k if k else v]
        total, run, nucleus = sum(prob[i] for i in left), 0.0, []
        for i in left:
            if nucleus and p < 1 and run >= p * total - 1e-12:
                break
            nucleus.append(i)
            run += prob[i]
        final = [i for i in nucleus if prob[i] >= m * prob.max() - 1e-12]
        mass = sum(prob[i] for i in final)
        seen = {}
        for u in (np.arange(400) + 0.5) / 400:
            tok, pr, stays, margin = ot.truncated_sample(x, t, k, p, m, u)
            assert sorted(np.nonzero(stays)[0]) == sorted(final)
            seen[tok] = seen.get(tok, 0) + 1
            assert abs(pr - prob[tok] / mass) < 1e-12
        for i in range(v):                                     # the draw is the inverse of the distribution
            assert abs(seen.get(i, 0) / 400 - (prob[i] / mass if i in final else 0.0)) <= 2 / 400
    assert ot.truncated_sample([1.0, 3.0, 3.0], 0, 0, 1.0, 0.0, 0.9)[0] == 1
