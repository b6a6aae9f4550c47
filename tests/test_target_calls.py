"""Calls of the target's side that end on the host: empty batches, limits, and what the binding refuses.  No GPU."""
import types

import pytest
import torch

import block_drafter_pos_gb300 as bd
from test_target_host import P, FakeHandle, _attn, _cache, _rows

b = bd.binding


def test_an_empty_batch_needs_no_addresses():
    """The lengths and the page table of no requests are empty tensors, whose address is 0."""
    h, r = FakeHandle(), _rows()
    for c in (_cache(page_table=None), _cache(page_table=None, max_pages=0, table_stride=0)):
        for f in (bd.lib().dflash2_paged_write, bd.lib().dflash2_paged_read):
            assert f(h.p, c, 0, 3, P, None, r, r, None, None) == b.OK
            assert f(h.p, c, 0, 0, P, None, _rows(p=None), _rows(p=None), None, None) == b.OK
            assert f(h.p, c, 0, -1, P, None, r, r, None, None) == b.E_INVAL
        assert bd.lib().dflash2_paged_attention(h.p, c, _attn(n_req=0, kv_len=None), None) == b.OK
        assert bd.lib().dflash2_paged_attention(h.p, c, _attn(n_req=0, kv_len=None, scale=float("nan")), None) == b.E_INVAL
    assert bd.lib().dflash2_paged_attention(h.p, None, _attn(n_req=0), None) == b.E_INVAL


def test_more_rows_than_32_bits_count_are_refused():
    """New tokens times the query heads of a KV head (4 here)."""
    f, h, c = bd.lib().dflash2_paged_attention, FakeHandle(), _cache()
    for n in (1 << 30, (1 << 31) - 1, (1 << 29) - 63):
        assert f(h.p, c, _attn(n_tokens=n, max_new=n), None) == b.E_UNSUPPORTED


@pytest.mark.parametrize("kind,off", [(b.T_F32, 2), (b.T_F32, 1), (b.T_BF16, 1), (b.T_F16, 3)])
def test_logits_off_their_types_alignment_are_refused(kind, off):
    a = b.SampleArgs(2, 100, kind, 0, P + off, 100, P, P, P, P, P, P, P, 4 * P, 100, P)
    assert bd.lib().dflash2_sample(a, None) == b.E_INVAL


# ----------------------------------------------------------------------------- the binding

def test_destroy_takes_live_handles_only(monkeypatch):
    """A handle destroyed before, or no handle at all, does not reach the library."""
    gone = []

    class Lib:
        @staticmethod
        def dflash2_paged_destroy(h):
            gone.append(h)
            return b.OK

    monkeypatch.setattr(b, "lib", lambda: Lib)
    monkeypatch.setitem(b._paged_cfg, 4096, ((b.KV_INT8, 16, 2, 128), 8, 0))
    bd.dflash2_paged_destroy(4096)
    for h in (4096, 4097, None):
        with pytest.raises(bd.Dflash2Error):
            bd.dflash2_paged_destroy(h)
    assert gone == [4096]


class Stub:
    """What the binding looks at of a tensor: here one of a given device."""

    def __init__(self, device, dtype, *shape):
        self.device_id, self.dtype, self.shape = device, dtype, torch.Size(shape)
        self.is_cuda = device >= 0
        self._stride = torch.empty(shape, dtype=torch.uint8).stride()

    def get_device(self):
        return self.device_id

    def stride(self, i=None):
        return self._stride if i is None else self._stride[i]

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return P


@pytest.fixture
def calls(monkeypatch):
    """The library's entry points replaced by one that notes the call; the current device is the first entry."""
    made, current = [], [0]
    real = b._calls()
    note = lambda *a: made.append(a) or b.OK  # noqa: E731
    fake = types.SimpleNamespace(int32=torch.int32, int64=torch.int64, float32=torch.float32, _C=types.SimpleNamespace(
        _cuda_getDevice=lambda: current[0], _cuda_getCurrentRawStream=lambda d: 77 + d))
    monkeypatch.setattr(b, "_fast", (fake,) + real[1:3] + (note,) * 4)
    monkeypatch.setitem(b._paged_cfg, 4096, ((b.KV_INT8, 16, 2, 128), 8, 0))
    return made, current


def _pool(dev=0, **other):
    d = lambda name: other.get(name, dev)  # noqa: E731
    f32, i8 = torch.float32, torch.int8
    return bd.paged_cache(Stub(d("k"), i8, 9, 16, 2, 128), Stub(d("v"), i8, 9, 16, 2, 128), Stub(d("table"), torch.int32, 3, 4),
                          Stub(d("k_scale"), f32, 9, 16, 2), Stub(d("v_scale"), f32, 9, 16, 2))


PAGED = dict(k=(torch.bfloat16, 6, 2, 128), v=(torch.bfloat16, 6, 2, 128), begin=(torch.int32, 4), kv_len=(torch.int32, 3),
             status=(torch.int32, 3), q=(torch.bfloat16, 6, 8, 128), out=(torch.bfloat16, 6, 8, 128), tree=(torch.int64, 6),
             lse=(torch.float32, 6, 8))
SAMPLE = dict(logits=(torch.float32, 2, 50), temperature=(torch.float32, 2), top_k=(torch.int32, 2), top_p=(torch.float32, 2),
              min_p=(torch.float32, 2), uniform=(torch.float32, 2), token=(torch.int32, 2), prob=(torch.float32, 2),
              kept=(torch.float32, 2, 50), status=(torch.int32, 2))


def _paged_calls(cache, dev=0, stream=None, **other):
    t = {k: Stub(other.get(k, dev), *v) for k, v in PAGED.items()}
    yield {"k", "v", "begin", "kv_len", "status"}, lambda: bd.dflash2_paged_write(
        4096, cache, t["k"], t["v"], t["begin"], t["kv_len"], t["status"], stream)
    yield {"k", "v", "begin", "kv_len", "status"}, lambda: bd.dflash2_paged_read(
        4096, cache, t["k"], t["v"], t["begin"], t["kv_len"], t["status"], stream)
    yield {"q", "out", "begin", "kv_len", "tree", "lse", "status"}, lambda: bd.dflash2_paged_attention(
        4096, cache, t["q"], t["out"], t["begin"], t["kv_len"], 6, 64, 0.1, tree_mask=t["tree"], lse=t["lse"],
        status=t["status"], stream=stream)


def _sample_call(dev=0, stream=None, **other):
    t = {k: Stub(other.get(k, dev), *v) for k, v in SAMPLE.items()}
    return bd.dflash2_sample(*(t[k] for k in ("logits", "temperature", "top_k", "top_p", "min_p", "uniform", "token")),
                             prob=t["prob"], kept=t["kept"], status=t["status"], stream=stream)


def test_calls_on_one_device_go_through(calls):
    made, _ = calls
    for _, call in _paged_calls(_pool()):
        call()
    _sample_call()
    assert len(made) == 4 and all(m[-1] == 77 for m in made)
    stream = types.SimpleNamespace(device_index=0, cuda_stream=5)
    for _, call in _paged_calls(_pool(), stream=stream):
        call()
    _sample_call(stream=stream)
    assert len(made) == 8 and all(m[-1] == 5 for m in made[4:])


@pytest.mark.parametrize("where", [1, -1])
def test_tensors_of_several_devices_are_refused(calls, where):
    made, _ = calls
    for name in ("k", "v", "table", "k_scale", "v_scale"):
        with pytest.raises(bd.Dflash2Error):
            _pool(**{name: where})
    for name in PAGED:
        for takes, call in _paged_calls(_pool(), **{name: where}):
            if name in takes:
                with pytest.raises(bd.Dflash2Error, match="device 0"):
                    call()
            else:
                call()
    assert len(made) == sum(name not in takes for name in PAGED for takes, _ in _paged_calls(_pool()))
    made.clear()
    for name in SAMPLE:
        with pytest.raises(bd.Dflash2Error):
            _sample_call(**{name: where})
    assert not made


def test_another_device_than_the_handles_or_the_current_one_is_refused(calls):
    made, current = calls
    for _, call in _paged_calls(_pool(1), 1):                  # pools and rows together on another device than the handle
        with pytest.raises(bd.Dflash2Error, match="handle on 0"):
            call()
    other = types.SimpleNamespace(device_index=1, cuda_stream=5)
    for stream in (None, other):
        current[0] = 1 if stream is None else 0                # a launch would go elsewhere
        for _, call in _paged_calls(_pool(), stream=stream):
            with pytest.raises(bd.Dflash2Error, match="current"):
                call()
        with pytest.raises(bd.Dflash2Error, match="current"):
            _sample_call(stream=stream)
    assert not made
    current[0] = 1
    _sample_call(1)
    assert len(made) == 1 and made[0][-1] == 78
