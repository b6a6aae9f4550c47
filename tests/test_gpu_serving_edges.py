"""Serving many samples of one prompt: calls at the edges of what they allow."""
import pytest
import torch

import block_drafter_pos_gb300 as bd
from test_gpu_serving import SharedSetup, check_shared, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("how,n,new", [("together", 4, 1), ("together", 4, 20), ("apart", 4, 1), ("auto", 70, 1)])
def test_groups_of_no_new_tokens_at_most(how, n, new):
    """max_group 0: every group that has rows breaks it, so all requests are flagged and no row is written; the next calls run."""
    s = SharedSetup([new] * n, [1000 + new + r for r in range(n)], hq=8, hk=4, dim=128, fmt="bf16", page=64, seed=1).share([n], [1000])
    assert how != "auto" or (n - 1) * 1000 * 2048 > 100 << 20    # (two launches)
    q = s.queries("bf16")
    out, status = torch.full_like(q, 7).cuda(), i32([0] * n)
    _, lse = s.attend_shared(q, out=out, status=status, how=how, max_group=0)
    assert status.tolist() == [1] * n and bool((out == 7).all()) and bool(lse.isnan().all())
    plan, rows = bd.make_rope(16), torch.ones(3, 1, 16, device="cuda")
    bd.dflash2_rope(plan, rows, rows, i32([0, 0, 0]))              # (an error left behind would be this call's)
    assert bool((rows == 1).all())
    status.zero_()
    out, lse = s.attend_shared(q, status=status, how=how)
    assert not status.any()
    check_shared(s, q, out, lse)
    s.close()


def test_rope_of_rows_in_any_order_but_onto_each_other():
    """Expanded rows are read, never written; rows of out may lie in any order in which they do not overlap."""
    plan, n, heads, dim = bd.make_rope(32), 3, 4, 32
    g = torch.Generator(device="cuda").manual_seed(0)
    x, pos = torch.randn(n, heads, dim, generator=g, device="cuda"), i32([5, 0, 1000])
    want = torch.empty_like(x)
    bd.dflash2_rope(plan, x, want, pos)
    for t, h in ((heads * dim, dim), (dim, n * dim), (160, 96), (40, 160), (96, 320), (dim, 3 * dim + 16)):
        room = torch.full((2000,), 7.0, device="cuda")
        out = room.as_strided((n, heads, dim), (t, h, 1))
        bd.dflash2_rope(plan, x, out, pos)
        assert torch.equal(out, want) and int((room != 7).sum()) <= x.numel()
        out.copy_(x)
        bd.dflash2_rope(plan, out, out, pos)
        assert torch.equal(out, want)
    one = x[:1].expand(n, heads, dim)
    bd.dflash2_rope(plan, one, want, pos)
    bd.dflash2_rope(plan, one.contiguous(), x, pos)
    assert torch.equal(x, want)
    for bad in (one, x[:, :1].expand(n, heads, dim), torch.zeros(500, device="cuda").as_strided((n, heads, dim), (64, 16, 1))):
        for source in (x, bad):
            with pytest.raises(bd.Dflash2Error):
                bd.dflash2_rope(plan, source, bad, pos)
        with pytest.raises(bd.Dflash2Error):
            bd.dflash2_rope(plan, x, want, pos, k=bad, k_out=bad)
