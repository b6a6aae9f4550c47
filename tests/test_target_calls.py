"""Calls of the target's side that end on the host: empty batches, limits, and what the binding refuses.  No GPU."""
import pytest

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
    monkeypatch.setitem(b._paged_cfg, 4096, ((b.KV_INT8, 16, 2, 128), 8))
    bd.dflash2_paged_destroy(4096)
    for h in (4096, 4097, None):
        with pytest.raises(bd.Dflash2Error):
            bd.dflash2_paged_destroy(h)
    assert gone == [4096]
