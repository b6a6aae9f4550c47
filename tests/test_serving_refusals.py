"""Calls for many samples of one prompt that are refused before anything is launched (no GPU)."""
import pytest

import block_drafter_pos_gb300 as bd
from test_serving_host import I32, _call_rope, _call_write, _rotation, calls  # noqa: F401
from test_target_calls import Stub
from test_target_host import FakeHandle, P, _cache, _rows

b = bd.binding
FAR = 1 << 30


@pytest.mark.parametrize("kw", [dict(token_stride=0), dict(head_stride=0), dict(token_stride=128), dict(token_stride=-128),
                                dict(token_stride=0, head_stride=0), dict(head_stride=64), dict(head_stride=-120),
                                dict(token_stride=384, head_stride=256 + 64), dict(token_stride=128, head_stride=128)])
def test_rows_turned_onto_each_other_are_refused(kw):
    """4 tokens of 2 heads of 128 (of 8 for queries): in place, or out of rows that are apart."""
    x = _rows(**kw)
    assert _call_rope(_rotation(), x=x, out=x) == b.E_INVAL
    assert _call_rope(_rotation(), x=_rows(), out=_rows(**{**kw, "p": FAR})) == b.E_INVAL
    assert _call_rope(_rotation(), x=_rows(), out=_rows(p=FAR), k_heads=2, k=_rows(p=2 * FAR), k_out=_rows(**{**kw, "p": 3 * FAR})) == b.E_INVAL
    h, r = FakeHandle(), _rows(p=FAR)
    q = _rows(**{"token_stride": 1024, **kw})
    assert _call_write(h.p, _rotation(), _cache(), q=q, q_out=q, k=r, v=r) == b.E_INVAL


def test_a_pool_of_another_page_size_than_the_handles_is_refused(calls):  # noqa: F811
    """The handle's pages have 16 positions, on device 0."""
    table, ref = Stub(0, I32, 3, 4), Stub(0, I32, 9)
    assert bd.page_pool(table, ref, 16, 4096).raw == bd.page_pool(table, ref, 16).raw
    for size, h, t in ((24, 4096, table), (8, 4096, table), (16, 4097, table), (16, 4096, Stub(1, I32, 3, 4))):
        with pytest.raises(bd.Dflash2Error):
            bd.page_pool(t, ref, size, h)
