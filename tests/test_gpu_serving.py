"""The calls for many samples of one prompt on the GPU, against the oracle: rotary positions, the pages of a pool, a tree's kept
tokens, and attention over shared prefixes."""
import numpy as np
import pytest
import torch

import block_drafter_pos_gb300 as bd
from oracle import serving as os_
from oracle import target as ot
from test_gpu_target import DT, HALF, Setup, check_attention

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


# ----------------------------------------------------------------------------- rotary positions

def rope_tolerance(want, reach, positions, rates, dtype):
    """Of a turned channel, in shares of |a| + |b| (times the amplitude): the angle, a fraction of a half turn rounded to fp32
    (2^-25 of pi), off by the plan's rounding of f / (2 pi) in FP64 (3 roundings and a cut, times the position); sine and
    cosine 2^-23 (an ulp); amplitude, product, product and sum 2^-24 each.  And the output's own rounding."""
    far = np.abs(np.asarray(positions, np.float64)).max(initial=0) * np.abs(rates).max() * 2.0 ** -51
    share = np.pi * 2.0 ** -25 + far + 2.0 ** -23 + 4 * 2.0 ** -24
    tiny = {"bf16": 2.0 ** -133, "fp16": 2.0 ** -25, "fp32": 2.0 ** -149}[dtype]
    return HALF[dtype] * np.abs(want) + share * (1 + HALF[dtype]) * reach + tiny


def check_rope(got, x, positions, rates, amplitude, interleaved, inverse, dtype):
    want, reach = os_.rope(x.cpu().float().numpy(), positions, rates, amplitude, interleaved, inverse)
    g = got.cpu().float().double().numpy()
    still = reach == 0
    # channels that are not turned pass bit for bit
    assert np.array_equal(g[..., 2 * len(rates):], want[..., 2 * len(rates):])
    bad = np.abs(g - want) > rope_tolerance(want, reach, positions, rates, dtype)
    assert not bad[~still].any(), np.abs(g - want)[bad].max()


SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="yarn", factor=4.0, original_len=32768, theta=1e6)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("dim,rot,interleaved,kw", [(128, 128, False, {}), (64, 16, True, SCALINGS[1]), (128, 96, False, SCALINGS[2]),
                                                    (80, 80, True, {}), (72, 48, False, SCALINGS[1]), (256, 256, False, SCALINGS[2]),
                                                    (576, 64, True, {}), (1024, 16, False, {})])
def test_rope_rows(dtype, dim, rot, interleaved, kw):
    """Counts from one token to many CTAs, strided rows both ways, positions near and far, either direction; rows beside
    them stay as they were."""
    plan = bd.make_rope(rot, interleaved=interleaved, **kw)
    rates, amplitude = os_.rope_rates(rot, **dict(dict(theta=1e7), **kw))
    for n, hx, hk, inverse in ((1, 1, 1, False), (5, 3, 2, True), (2, 9, 0, False), (1300, 2, 1, True)):
        g = np.random.default_rng(n + dim)
        pos = g.integers(0, 200000, n)
        pos[:1] = 0
        wide = torch.from_numpy(g.standard_normal((n, hx + hk + 2, dim)).astype(np.float32)).to(DT[dtype]).cuda()
        x, k = wide[:, 1:1 + hx], wide[:, 1 + hx:1 + hx + hk]               # views of one projection
        out = torch.full((hx + 1, n, dim), 7.0, dtype=DT[dtype], device="cuda").transpose(0, 1)   # heads outside tokens
        k_out = torch.full((n, hk + 1, dim + 64 // DT[dtype].itemsize), 7.0, dtype=DT[dtype], device="cuda")
        pair = dict(k=k, k_out=k_out[:, :hk, :dim]) if hk else {}
        bd.dflash2_rope(plan, x, out[:, :hx], i32(pos), inverse=inverse, **pair)
        torch.cuda.synchronize()
        check_rope(out[:, :hx], x, pos, rates, amplitude, interleaved, inverse, dtype)
        assert bool((out[:, hx:] == 7).all()) and bool((k_out[:, hk:] == 7).all()) and bool((k_out[..., dim:] == 7).all())
        if hk:
            check_rope(k_out[:, :hk, :dim], k, pos, rates, amplitude, interleaved, inverse, dtype)
        # in place: the same bits, and nothing beside the rows
        before = wide.clone()
        bd.dflash2_rope(plan, x, x, i32(pos), inverse=inverse, **(dict(k=k, k_out=k) if hk else {}))
        torch.cuda.synchronize()
        assert torch.equal(x, out[:, :hx]) and torch.equal(k, k_out[:, :hk, :dim])
        assert torch.equal(wide[:, 0], before[:, 0]) and torch.equal(wide[:, -1], before[:, -1])


def test_rope_at_the_ends_of_the_positions():
    """Any int32 position, negative ones and fast pairs included."""
    pos = np.array([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 123456789, -987654321])
    rates = np.array([1.0, -0.3, 5.0, 1e-9, 0.0, 2.5, 1e-4, 100.0])
    plan = bd.make_rope(16, scaling="table", table=list(rates), amplitude=0.5)
    x = torch.randn(8, 2, 16, generator=torch.Generator().manual_seed(0)).cuda()
    out = torch.empty_like(x)
    bd.dflash2_rope(plan, x, out, i32(pos))
    check_rope(out, x, pos, rates, 0.5, False, False, "fp32")


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_gradient(interleaved):
    """The inverse's rows are the gradient: against the transposed matrix of the call itself, column by column (it is
    linear), and against differences."""
    rot, dim, n = 48, 64, 3
    plan = bd.make_rope(rot, 1e4, interleaved=interleaved, scaling="yarn", factor=8.0, original_len=100)
    pos = i32([5, 77, 4000])
    eye = torch.eye(dim, device="cuda")[None].expand(n, dim, dim).contiguous()      # head j of a token: unit vector j
    cols, rows = torch.empty_like(eye), torch.empty_like(eye)
    bd.dflash2_rope(plan, eye, cols, pos)                                           # cols[t, j] = R e_j
    bd.dflash2_rope(plan, eye, rows, pos, inverse=True)                             # rows[t, i] = R^T e_i
    # both are cosines and sines of the same fp32 angle, whose sine is odd: products with 0 and 1 are exact
    assert torch.equal(rows, cols.transpose(1, 2))
    g = torch.Generator(device="cuda").manual_seed(1)
    x, gy = (torch.randn(n, 4, dim, generator=g, device="cuda") for _ in "xg")
    gx = torch.empty_like(x)
    bd.dflash2_rope(plan, gy, gx, pos, inverse=True)
    y1, y0, h = torch.empty_like(x), torch.empty_like(x), 0.5
    for _ in range(4):
        d = torch.randn(x.shape, generator=g, device="cuda")
        bd.dflash2_rope(plan, x + h * d, y1, pos)
        bd.dflash2_rope(plan, x - h * d, y0, pos)
        diff = float(((y1 - y0).double() * gy.double()).sum() / (2 * h))
        want = float((gx.double() * d.double()).sum())
        # of each of 768 products' factors: the sums' and the rotation's roundings, under 2^-20 of (|x| + |d|) |gy| in all
        assert abs(diff - want) <= 2.0 ** -19 * 2 * float(((x.abs() + d.abs()).double() * gy.abs().double()).sum())


def test_rope_passes_what_is_not_finite():
    x = torch.zeros(2, 1, 32, device="cuda")
    x[0, 0, 3], x[1, 0, 30] = float("nan"), float("inf")
    out = torch.empty_like(x)
    bd.dflash2_rope(bd.make_rope(16), x, out, i32([0, 9]))
    bad = (~torch.isfinite(out)).nonzero().tolist()
    assert bad == [[0, 0, 3], [0, 0, 11], [1, 0, 30]]


@pytest.mark.parametrize("fmt", ["bf16", "fp16", "int8", "e4m3"])
@pytest.mark.parametrize("dim,rot,interleaved,src,order,page", [(128, 128, False, "bf16", "pch", 16), (64, 32, True, "fp16", "phc", 1),
                                                                (128, 48, False, "fp32", "hpc", 24), (64, 64, False, "bf16", "phc", 64),
                                                                (128, 112, True, "fp32", "pch", 7)])
def test_rope_write(fmt, dim, rot, interleaved, src, order, page):
    """Turned queries, and what the cache holds of turned keys: off by the rotation's error and half a step of the format; values
    as dflash2_paged_write stores them; other rows of the pool as they were."""
    new, length = [3, 0, 1, 17, 40], [3, 9, 1000, 30, 41]
    s = Setup(new, length, hq=6, hk=3, dim=dim, page=page, fmt=fmt, order=order, seed=dim + page)
    kw = SCALINGS[2]
    plan = bd.make_rope(rot, interleaved=interleaved, **kw)
    rates, amplitude = os_.rope_rates(rot, **kw)
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(s.tokens, h, dim, generator=g).to(DT[src]).cuda() for h in (6, 3, 3))
    pos = np.concatenate([np.arange(t - n, t) for n, t in zip(new, length)])
    before = [t.clone() for t in (s.gk, s.gv)]
    touched = torch.zeros(s.gk.shape[:2], dtype=torch.bool)
    for r in range(5):
        for p in range(length[r] - new[r], length[r]):
            touched[s.table[r, p // page], p % page] = True
    for given in (None, np.random.default_rng(1).integers(0, 100000, s.tokens)):
        at = pos if given is None else given
        status = torch.zeros(5, dtype=torch.int32, device="cuda")
        q_out = torch.full_like(q, 7)
        args = (s.begin, s.kv_len, None if given is None else i32(given), status)
        bd.dflash2_paged_rope_write(s.handle, plan, s.cache, q, q_out, k, v, *args)
        kr, vr = (torch.empty(s.tokens, 3, dim, device="cuda") for _ in "kv")
        bd.dflash2_paged_read(s.handle, s.cache, kr, vr, s.begin, s.kv_len)
        torch.cuda.synchronize()
        assert not status.any()
        check_rope(q_out, q, at, rates, amplitude, interleaved, False, src)
        want, reach = os_.rope(k.cpu().float().numpy(), at, rates, amplitude, interleaved)
        off = rope_tolerance(want, reach, at, rates, "fp32")
        got = kr.double().cpu().numpy()
        if fmt in ot.QMAX:
            top = (np.abs(want) + off).max(-1, keepdims=True)
            step = top / 127 / 2 if fmt == "int8" else np.maximum(2.0 ** -4 * (np.abs(want) + off), top / 448 * 2.0 ** -10)
            # (the scale's, the quotient's and the read value's roundings, 2^-24 each of at most the row's largest; the top itself
            # may move by `off`)
            tol = step * 1.001 + 2 * off + off.max(-1, keepdims=True) + 4 * 2.0 ** -24 * top
        else:
            tol = HALF[fmt] * (np.abs(want) + off) + off + 2.0 ** -25
        assert (np.abs(got - want) <= tol).all(), np.abs(got - want).max()
        # values: as dflash2_paged_write stores them
        if fmt in ot.QMAX:
            codes, scale = ot.quantise(v.cpu().float().numpy(), fmt)
            assert np.array_equal(vr.cpu().numpy(), (codes.astype(np.float32) * scale[..., None]).astype(np.float32))
        else:
            assert torch.equal(vr, v.to(DT[fmt]).float())
        for pool, old in zip((s.gk, s.gv), before):
            a, c = (t.contiguous().view(torch.uint8).cpu().view(*t.shape[:3], -1) for t in (pool, old))
            assert torch.equal(a[~touched], c[~touched])
        # in place and without queries: the same
        held = [t.clone() for t in (s.gk, s.gv)]
        s.gk.copy_(before[0])
        q2 = q.clone()
        bd.dflash2_paged_rope_write(s.handle, plan, s.cache, q2, q2, k, v, *args)
        assert torch.equal(q2, q_out) and torch.equal(s.gk.contiguous().view(torch.uint8), held[0].contiguous().view(torch.uint8))
        s.gk.copy_(before[0])
        bd.dflash2_paged_rope_write(s.handle, plan, s.cache, None, None, k, v, *args)
        assert torch.equal(s.gk.contiguous().view(torch.uint8), held[0].contiguous().view(torch.uint8))
    s.close()


def test_rope_write_flags_bad_requests():
    """Bad lengths and ranges touch nothing (queries included); a bad page's keys are not written."""
    s = Setup([4, 4, 4, 4], [20, 20, 20, 20], fmt="int8", page=16)
    s.gtable[1, 1] = s.gk.shape[0]                         # past the pool
    s.kv_len[2] = 2                                        # fewer positions than new tokens
    s.kv_len[3] = 2 * 16 + 1                               # past the page table's row
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k = (torch.randn(16, h, 128, generator=g, device="cuda", dtype=torch.bfloat16) for h in (4, 2))
    before, q_out = s.gk.clone(), torch.full_like(q, 7)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    bd.dflash2_paged_rope_write(s.handle, bd.make_rope(128), s.cache, q, q_out, k, k, s.begin, s.kv_len, status=status)
    assert status.tolist() == [0, 1, 1, 1]
    assert bool((q_out[8:] == 7).all()) and not bool((q_out[:8] == 7).all(-1).any())
    changed = (s.gk != before).flatten(2).any(-1)
    assert changed.nonzero().tolist() == [[int(s.table[0, 1]), i] for i in range(4)]
    s.close()


# ----------------------------------------------------------------------------- the pages of a pool

class Pages:
    """A pool's state on the GPU beside the oracle's."""

    def __init__(self, rows, width, n_pages, page, stride=None):
        self.page, self.n = page, rows
        self.wide = torch.full((rows, stride or width), -1, dtype=torch.int32, device="cuda")
        self.table, self.ref = self.wide[:, :width], torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        self.kv = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.copies = torch.full((3, rows), 99, dtype=torch.int32, device="cuda")
        self.pool = bd.page_pool(self.table, self.ref, page)
        self.want = ([[-1] * width for _ in range(rows)], [0] * n_pages, [0] * rows)

    def check(self, *, leak=True):
        torch.cuda.synchronize()
        assert self.kv.tolist() == self.want[2]
        assert self.table.tolist() == self.want[0]
        assert self.ref.tolist() == self.want[1]
        if leak:                                           # the counts are what the table says
            held = np.zeros(self.ref.numel(), int)
            for row, length in zip(self.want[0], self.want[2]):
                for t in row[:-(-length // self.page)]:
                    held[t] += 1
                assert all(t == -1 for t in row[-(-length // self.page):])
            assert np.array_equal(held, self.want[1])

    def resize(self, new, leak=True):
        copies, status = os_.pages_resize(*self.want, new, self.page)
        st = torch.zeros(self.n, dtype=torch.int32, device="cuda")
        bd.dflash2_pages_resize(self.pool, self.kv, i32(new), self.copies, st)
        self.check(leak=leak)
        assert self.copies.T.tolist() == [list(c) for c in copies] and st.tolist() == status
        return copies, status

    def fork(self, parent, child, leak=True):
        status = os_.pages_fork(*self.want, parent, child, self.page)
        st = torch.zeros(len(parent), dtype=torch.int32, device="cuda")
        bd.dflash2_pages_fork(self.pool, i32(parent), i32(child), self.kv, st)
        self.check(leak=leak)
        assert st.tolist() == status
        return status


@pytest.mark.parametrize("rows,width,n_pages,page,seed", [(1, 3, 4, 1, 0), (7, 12, 60, 4, 1), (33, 9, 200, 16, 2), (40, 30, 1025, 3, 3),
                                                          (300, 5, 5000, 24, 4), (1024, 2, 3000, 8, 5)])
def test_pages_in_a_random_life(rows, width, n_pages, page, seed):
    """Rows grow, are cut, freed and forked at random, in a pool that runs short; every state, copy and status is the oracle's."""
    g = np.random.default_rng(seed)
    p = Pages(rows, width, n_pages, page, stride=width + 3)
    seen = set()
    for step in range(12):
        kv = np.array(p.want[2])
        move = g.integers(0, 4, rows)
        new = np.where(move == 0, 0, np.where(move == 1, kv, np.where(move == 2, kv // 2, np.minimum(kv + g.integers(0, 3 * page, rows), width * page))))
        if step % 5 == 4:
            new = np.minimum(new, kv // 3)                 # make room
        copies, status = p.resize(new.tolist())
        seen |= set(status) | {-1 for c in copies if c[0] >= 0}
        kv = np.array(p.want[2])
        free, held = [list(g.permutation(np.nonzero(m)[0])) for m in (kv == 0, kv > 0)]
        if free and held:
            n = int(g.integers(1, min(len(free), 8) + 1))
            assert p.fork([int(held[int(g.integers(0, min(2, len(held))))]) for _ in range(n)], [int(c) for c in free[:n]]) == [0] * n
    p.resize([0] * rows)
    assert not p.ref.any() and bool((p.table == -1).all()) and bool((p.wide[:, width:] == -1).all())
    assert rows == 1 or -1 in seen                         # copies on write were among them


def test_pages_sharers_that_all_grow():
    """The first keeps the page if every holder grows; not if one stays, is cut, or is out of bounds."""
    for others, kept in (([9, 9, 9], True), ([9, 6, 9], False), ([9, 3, 9], False), ([9, 0, 9], False)):
        p = Pages(4, 4, 30, 4)
        p.resize([6, 0, 0, 0])
        p.fork([0, 0, 0], [1, 2, 3])
        copies, _ = p.resize([7] + others)
        assert (copies[0][0] < 0) == kept and copies[1][0] >= 0


def test_pages_that_run_out():
    """Rows are served in order until one does not fit; those that take nothing go on."""
    p = Pages(5, 4, 6, 4)
    assert p.resize([8, 8, 12, 4, 0])[1] == [0, 0, 5, 5, 0]
    assert p.resize([8, 4, 12, 0, 0])[1] == [0, 0, 5, 0, 0]         # (what row 1 gives back is free to the next call)
    assert p.resize([8, 4, 12, 0, 0])[1] == [0] * 5
    assert p.resize([9, 5, 13, 1, 1])[1] == [5, 5, 5, 5, 5]


def test_pages_in_a_large_pool():
    """4,194,304 pages (the most), all but a few held, free ones at both ends and at chunks' borders."""
    n = 1 << 22
    p = Pages(3, 8, n, 16)
    p.ref.fill_(1)
    free = [0, 31, 32, 1023, 1024, 8191, 8192, 8193, 1 << 20, n - 1025, n - 2, n - 1]
    p.ref[torch.tensor(free, device="cuda")] = 0
    st = torch.zeros(3, dtype=torch.int32, device="cuda")
    bd.dflash2_pages_resize(p.pool, p.kv, i32([70, 16, 90]), p.copies, st)
    assert p.table[0, :5].tolist() == free[:5] and p.table[1, :1].tolist() == free[5:6] and p.table[2, :6].tolist() == free[6:]
    assert bool((p.ref == 1).all()) and not st.any()
    bd.dflash2_pages_resize(p.pool, p.kv, i32([70, 17, 90]), p.copies, st)
    assert st.tolist() == [0, 5, 0] and p.kv.tolist() == [70, 16, 90]
    bd.dflash2_pages_resize(p.pool, p.kv, i32([0, 0, 0]), p.copies, None)
    assert (p.ref == 0).nonzero().flatten().tolist() == free


def test_pages_flag_bad_rows():
    """Lengths and page ids out of bounds: flagged, nothing taken, other rows served."""
    p = Pages(6, 3, 20, 4)
    p.resize([6, 6, 6, 6, 5, 6])
    p.table[1, 1] = p.want[0][1][1] = 20                    # past the pool, and negative: tails of rows that grow
    p.table[2, 1] = p.want[0][2][1] = -3
    p.table[3, 0] = p.want[0][3][0] = 1 << 30               # in a row that is cut to nothing
    hole = p.want[0][4][1]
    p.ref[hole] = p.want[1][hole] = 0                       # a held page without a holder
    assert p.resize([7, 7, 7, 0, 7, 13], leak=False)[1] == [0, 1, 1, 1, 1, 1]
    assert p.resize([-1, -5, 6, 2, 5, 6], leak=False)[1] == [1, 1, 0, 0, 0, 0]
    q = Pages(4, 3, 20, 4)
    q.resize([6, 5, 0, 0])
    assert q.fork([0, -1, 4, 0, 0], [2, 3, 3, 4, -1]) == [0, 1, 1, 1, 1]
    q.resize([6, 5, 0, 0])
    assert q.fork([0, 1], [2, 2]) == [1, 1]                 # a child twice
    assert q.fork([0, 2], [2, 3]) == [1, 1]                 # a parent that is a child
    assert q.fork([0], [1]) == [1] and q.fork([3], [3]) == [1]
    q.table[0, 1] = q.want[0][0][1] = 20
    assert q.fork([0, 1], [2, 3], leak=False) == [1, 0]
    q.kv[0] = q.want[2][0] = 13
    assert q.fork([0], [2], leak=False) == [1]


@pytest.mark.parametrize("fmt", ["bf16", "fp16", "int8", "e4m3"])
@pytest.mark.parametrize("hk,dim,page,order", [(2, 128, 16, "phc"), (3, 64, 1, "pch"), (8, 128, 64, "pch"), (1, 64, 24, "hpc")])
def test_pages_copy(fmt, hk, dim, page, order):
    """Codes and scales bit for bit in every layer (30: two launches), the first positions of a page alone; entries out of bounds are
    flagged, negative ones passed over."""
    layers = [Setup([1], [5 * page], hq=hk, hk=hk, dim=dim, page=page, fmt=fmt, order=order, seed=x) for x in range(3)]
    pools = [[t for t in (s.gk, s.gv, s.gks, s.gvs) if t is not None] for s in layers]
    before = [[t.clone() for t in p] for p in pools]
    n = layers[0].gk.shape[0]
    lists = [[0, 5, -1, 2, 0, n, 2], [1, 3, 4, -7, 6, 4, n], [page, (page + 1) // 2, page, page, page + 1, page, 1]]
    status = torch.zeros(7, dtype=torch.int32, device="cuda")
    bd.dflash2_pages_copy(layers[0].handle, [s.cache for s in layers] * 10, i32(lists), status)
    torch.cuda.synchronize()
    assert status.tolist() == [0, 0, 0, 0, 1, 1, 1]
    for now, was in zip(pools, before):
        for a, c in zip(now, was):
            a, c = (t.contiguous().view(torch.uint8).cpu() for t in (a, c))
            want = c.clone()
            want[1], want[3, :(page + 1) // 2] = c[0], c[5, :(page + 1) // 2]
            assert torch.equal(a, want)
    for s in layers:
        s.close()


@pytest.mark.parametrize("fmt", ["bf16", "fp16", "int8", "e4m3"])
@pytest.mark.parametrize("hk,dim,page,order", [(2, 128, 16, "phc"), (3, 64, 1, "pch"), (8, 128, 64, "pch"), (1, 64, 24, "hpc")])
def test_kept_tokens(fmt, hk, dim, page, order):
    """Codes and scales bit for bit; everything else as it was; requests out of bounds flagged and untouched."""
    new, length = [33, 64, 1, 8, 40, 5, 5, 5, 5, 0], [40, 64, 300, 30, 100, 9, 9, 9, 9, 7]
    paths = [[0, 3, 4, 9, 20, 32], list(range(64)), [0], [], [0, 1, 2, 39], [0, 5], [1, 1], [2, 1], [0, 1], []]
    layers = [Setup(new, length, hq=hk, hk=hk, dim=dim, page=page, fmt=fmt, order=order, seed=x) for x in range(2)]
    most = 64
    keep = np.full((10, most + 5), -9, np.int32)
    for r, path in enumerate(paths):
        keep[r, :len(path)] = path
    n_keep = [len(x) for x in paths]
    n_keep[8] = 6                                          # more than there are
    wide = i32(keep)
    pools = [[t for t in (s.gk, s.gv, s.gks, s.gvs) if t is not None] for s in layers]
    before = [[t.contiguous().view(torch.uint8).cpu() for t in p] for p in pools]
    status, kv_out = torch.zeros(10, dtype=torch.int32, device="cuda"), torch.zeros(10, dtype=torch.int32, device="cuda")
    bd.dflash2_paged_keep(layers[0].handle, [s.cache for s in layers], layers[0].begin, layers[0].kv_len, wide[:, :most], i32(n_keep),
                          kv_out, status)
    torch.cuda.synchronize()
    bad = [5, 6, 7, 8]
    assert [r for r, x in enumerate(status.tolist()) if x] == bad
    assert kv_out.tolist() == [t if r in bad else t - n + len(p) for r, (n, t, p) in enumerate(zip(new, length, paths))]
    for s, now, was in zip(layers, pools, before):
        for a, c in zip(now, was):
            want = c.clone()
            for r, path in enumerate(paths):
                for j, x in enumerate(path if r not in bad else []):
                    src, dst = length[r] - new[r] + x, length[r] - new[r] + j
                    want[s.table[r, dst // page], dst % page] = c[s.table[r, src // page], src % page]
            assert torch.equal(a.contiguous().view(torch.uint8).cpu(), want)
    for s in layers:
        s.close()


def test_kept_tokens_in_many_layers_and_on_bad_pages():
    """Two launches of layers; a bad page in one layer leaves that layer's request alone, and the others move."""
    s = [Setup([9, 9], [20, 20], hq=2, hk=2, dim=64, page=4, fmt="bf16", seed=x) for x in range(26)]
    s[25].gtable[1, 4] = 1 << 20
    before = [x.gk.clone() for x in s]
    status, kv_out = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    bd.dflash2_paged_keep(s[0].handle, [x.cache for x in s], s[0].begin, s[0].kv_len, i32([[0, 8], [0, 8]]), i32([2, 2]), kv_out, status)
    assert status.tolist() == [0, 1] and kv_out.tolist() == [13, 13]
    for x, (setup, was) in enumerate(zip(s, before)):
        for r in range(2):
            moved = torch.equal(setup.gk[int(setup.table[r, 3]), 0], was[int(setup.table[r, 4]), 3])
            assert moved == (x < 25 or r == 0), (x, r)
        setup.close()


# ----------------------------------------------------------------------------- attention over shared prefixes

class SharedSetup(Setup):
    """Requests in groups: those behind a group's first one have no pages of the prefix of their own (their table's entries are
    not pages), and their rows of the page in which it ends hold NaN."""

    def share(self, sizes, prefix):
        self.sizes, self.prefix = sizes, prefix
        r = 0
        for size, p in zip(sizes, prefix):
            for x in range(r + 1, r + size):
                for side, pool, scales in ((0, self.gk, self.gks), (1, self.gv, self.gvs)):
                    rest = p % self.page
                    if rest:
                        page = int(self.table[x, p // self.page])
                        if scales is not None:
                            scales[page, :rest] = float("nan")
                        else:
                            pool[page, :rest] = float("nan")
                    self.vals[x][side] = np.concatenate([self.vals[r][side][:p], self.vals[x][side][p:]])
                self.gtable[x, :p // self.page] = -5
            r += size
        self.group_begin = i32(np.concatenate([[0], np.cumsum(sizes)]))
        self.prefix_len = i32(prefix)
        begins = np.concatenate([[0], np.cumsum(self.new)])
        edges = np.concatenate([[0], np.cumsum(sizes)])
        self.max_group = max([int(begins[b] - begins[a]) for a, b in zip(edges[:-1], edges[1:])] + [1])
        self.work = torch.full((bd.dflash2_paged_shared_bytes(self.handle, self.tokens),), 255, dtype=torch.uint8, device="cuda")
        return self

    def attend_shared(self, q, out=None, status=None, **kw):
        q = q.cuda()
        out = torch.full_like(q, float("nan")) if out is None else out
        lse = torch.full(q.shape[:2], float("nan"), device="cuda")
        kw.setdefault("max_group", self.max_group)
        kw.setdefault("max_prefix", max(self.prefix + [0]))
        kw.setdefault("scale", self.dim ** -0.5)
        kw.setdefault("how", "together")
        bd.dflash2_paged_attention_shared(self.handle, self.cache, q, out, self.begin, self.kv_len, self.group_begin, self.prefix_len,
                                          self.work, max_new=max(self.new + [1]), max_len=max(self.length + [1]), lse=lse, status=status, **kw)
        torch.cuda.synchronize()
        return out, lse


def check_shared(s, q, out, lse, **kw):
    """Against the single call's bound.  That counts a rescaling (2^-22) for every tile of 64 keys and two more, though one is due
    only where a maximum has grown by 2^8; the join is one such rescaling of either part."""
    check_attention(s, q, out, lse, **kw)


CASES = [  # sizes of groups, prefixes, new tokens, own keys
    ([3], [100], [1, 1, 1], [5, 1, 70]),                                          # few rows either way
    ([1], [64], [1], [1]),
    ([40], [517], [1] * 40, [1 + 13 * (r % 9) for r in range(40)]),               # many rows of a prefix, few of its own
    ([5, 0, 1, 6], [130, 7, 0, 257], [8] * 12, [8 + 31 * r for r in range(12)]),  # an empty group, one without a prefix
    ([2, 2], [1, 300], [70, 0, 65, 90], [70, 3, 200, 90]),                        # many rows either way; no new tokens
    ([12], [1000], [1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12], [400, 2, 3, 90, 5, 6, 7, 64, 63, 65, 11, 12]),
]


@pytest.mark.parametrize("fmt,qtype", [("bf16", "bf16"), ("fp16", "fp16"), ("int8", "bf16"), ("e4m3", "fp16")])
@pytest.mark.parametrize("hq,hk,dim,page,order", [(4, 2, 128, 16, "phc"), (3, 1, 64, 24, "hpc"), (16, 2, 128, 7, "pch")])
@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("how", ["together", "apart"])
def test_shared_attention(how, case, hq, hk, dim, page, order, fmt, qtype):
    sizes, prefix, new, own = CASES[case]
    pre = [p for n, p in zip(sizes, prefix) for _ in range(n)]
    s = SharedSetup(new, [p + n for p, n in zip(pre, own)], hq=hq, hk=hk, dim=dim, page=page, order=order, fmt=fmt,
                    seed=case + dim).share(sizes, prefix)
    q = s.queries(qtype, amp=2.0)
    status = torch.zeros(len(new), dtype=torch.int32, device="cuda")
    out, lse = s.attend_shared(q, status=status, how=how)
    assert not status.any()
    check_shared(s, q, out, lse)
    again, lse2 = s.attend_shared(q, how=how)              # the same bits, whatever the workspace held
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)
    if case in (0, 3):
        check_shared(s, q, *s.attend_shared(q, causal=False, how=how), causal=False)
        check_shared(s, q, *s.attend_shared(q, scale=-0.3, how=how), scale=-0.3)
    s.close()


def test_shared_attention_chooses_by_the_bytes():
    """On either side of the border the call's bits are those of the way it names: 15 requests read positions of 4 KB again;
    the border is 100 MiB for 16 rows and 200 MiB above."""
    for new, prefix, way in ((1, 1706, "apart"), (1, 1707, "together"), (8, 3413, "apart"), (8, 3414, "together")):
        s = SharedSetup([new] * 16, [prefix + new + 3 * r for r in range(16)], hq=32, hk=8, page=64, seed=prefix).share([16], [prefix])
        assert (15 * prefix * 4096 <= (100 << 20 if new == 1 else 200 << 20)) == (way == "apart")
        q = s.queries("bf16")
        ways = {w: s.attend_shared(q, how=w)[1] for w in ("auto", "together", "apart")}
        assert not torch.equal(ways["together"], ways["apart"])              # (joined in another order)
        assert torch.equal(ways["auto"], ways[way])
        s.close()


@pytest.mark.parametrize("fmt,qtype", [("bf16", "bf16"), ("e4m3", "bf16")])
@pytest.mark.parametrize("nodes", [3, 33, 64])
@pytest.mark.parametrize("how", ["together", "apart"])
def test_shared_attention_of_trees(how, fmt, qtype, nodes):
    """Tree masks; words without a bit leave a row with the prefix alone, or, without a prefix, with nothing."""
    sizes, prefix = [3, 2], [90, 0]
    new, own = [nodes] * 5, [nodes + 4, nodes, nodes + 70, nodes, nodes]
    s = SharedSetup(new, [p + n for p, n in zip([90] * 3 + [0] * 2, own)], fmt=fmt, seed=nodes).share(sizes, prefix)
    g = np.random.default_rng(nodes)
    tree = np.array([int(g.integers(0, 1 << 63)) | 1 << i for _ in range(5) for i in range(nodes)], np.uint64)
    tree[2] = tree[nodes + 1] = tree[3 * nodes] = 0
    q = s.queries(qtype)
    out, lse = s.attend_shared(q, tree_mask=torch.from_numpy(tree.view(np.int64)).cuda(), how=how)
    check_shared(s, q, out, lse, tree=tree)
    assert not out[3 * nodes].any() and bool((lse[3 * nodes] == -float("inf")).all())
    s.close()


def test_shared_attention_is_the_single_call():
    """The same requests through dflash2_paged_attention, each with the prefix's pages in its own row of the table."""
    sizes, prefix = [16], [2048]
    s = SharedSetup([4] * 16, [2048 + 4 + 100 * r for r in range(16)], hq=8, hk=2, page=32, fmt="int8").share(sizes, prefix)
    q = s.queries("bf16")
    out, lse = s.attend_shared(q)
    s.gtable[1:, :64] = s.gtable[0, :64]
    want, wl = s.attend(q)
    # each is within its bound of the exact result: half a step of the output (2^-8 of it, and of the sum of magnitudes), twice
    assert (out.float() - want.float()).abs().max() <= 2 * 2.0 ** -8 * want.float().abs().max()
    assert (lse - wl).abs().max() <= 2.0 ** -12
    s.close()


@pytest.mark.parametrize("how", ["together", "apart"])
def test_shared_attention_flags_bad_groups_and_requests(how):
    """A group or a request that breaks its bounds is flagged and its rows stay; the others are served."""
    sizes, prefix = [2, 2, 2], [100, 50, 70]
    new, length = [3] * 6, [110, 120, 60, 53, 90, 100]

    def fresh():
        s = SharedSetup(new, length, fmt="bf16", seed=3).share(sizes, prefix)
        q = s.queries("bf16")
        return s, q, torch.full_like(q, 7).cuda(), torch.zeros(6, dtype=torch.int32, device="cuda")

    def look(s, q, out, status, bad, **kw):
        out, lse = s.attend_shared(q, out=out, status=status, how=how, **kw)
        assert status.tolist() == [int(r in bad) for r in range(6)]
        for r in range(6):
            rows = out[3 * r:3 * r + 3]
            assert bool((rows == 7).all()) if r in bad else not bool((rows == 7).any())
        keep = [r for r in range(6) if r not in bad]
        check_shared(s, q, out, lse, skip=bad)
        s.close()
        return keep

    s, *x = fresh()
    s.prefix_len[1] = 51                                    # past a request's old positions: 53 - 3
    look(s, *x, bad=[3])
    s, *x = fresh()
    s.prefix_len[1] = 101                                   # past max_prefix
    look(s, *x, bad=[2, 3])
    s, *x = fresh()
    s.prefix_len[2] = -1
    look(s, *x, bad=[4, 5])
    s, *x = fresh()
    s.kv_len[0] = 102                                       # fewer old positions than the prefix
    look(s, *x, bad=[0])
    s, *x = fresh()
    s.kv_len[5] = -4
    look(s, *x, bad=[5])
    s, *x = fresh()
    look(s, *x, bad=[0, 1, 2, 3, 4, 5], max_group=5)        # groups of six tokens
    s, *x = fresh()
    for at, value in ((3, 5), (3, 7), (0, 1), (0, -1), (1, 1 << 30), (2, 1), (2, -(1 << 31))):
        s.group_begin[at] = value                           # not ascending from the first request to the last
        look(s, *x, bad=[0, 1, 2, 3, 4, 5])
        s, *x = fresh()
    s.begin[6] = 19                                         # past the rows
    look(s, *x, bad=[4, 5])


@pytest.mark.parametrize("how", ["together", "apart"])
def test_shared_attention_masks_bad_pages(how):
    """A bad page of the prefix is masked for the whole group, which is flagged; one behind it for its request."""
    sizes, prefix = [3, 1], [64, 0]
    s = SharedSetup([2] * 4, [90, 100, 70, 20], fmt="e4m3", page=16).share(sizes, prefix)
    s.gtable[0, 1] = 1 << 20
    s.gtable[1, 5] = -1
    q = s.queries("bf16")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    out, lse = s.attend_shared(q, status=status, how=how)
    assert status.tolist() == [1, 1, 1, 0]
    qd = q.double().numpy()
    for r in range(4):
        see = ot.visible(2, s.length[r])
        if r < 3:
            see[:, 16:32] = False
        if r == 1:
            see[:, 80:96] = False
        want, _, spread, _ = ot.paged_attention(qd[2 * r:2 * r + 2], *s.vals[r], s.dim ** -0.5, see)
        got = out[2 * r:2 * r + 2].double().cpu().numpy()
        # the output's rounding, a weight's to fp16 and under 2^-16 of the fp32 sums of short rows
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -15) * spread + 2.0 ** -20).all()
    s.close()


@pytest.mark.parametrize("how", ["together", "apart"])
def test_shared_attention_of_values_that_are_not_finite(how):
    """In the prefix they show in the group's rows alone; behind it in the rows that see them; in masked places nowhere."""
    s = SharedSetup([2, 2, 2], [200, 210, 40], fmt="bf16", page=16).share([2, 1], [128, 0])
    s.gv[int(s.table[0, 3]), 2, 1, 5] = float("inf")                # position 50 of the prefix
    s.vals[0][1][50, 1, 5] = s.vals[1][1][50, 1, 5] = np.inf
    s.gv[int(s.table[1, 209 // 16]), 209 % 16, 0, 9] = float("nan")  # the newest token of request 1
    s.vals[1][1][209, 0, 9] = np.nan
    q = s.queries("bf16")
    out, lse = s.attend_shared(q, how=how)
    bad = [tuple(x) for x in (~torch.isfinite(out)).nonzero().tolist()]
    assert {(t, h) for t, h, c in bad if c == 5} == {(t, h) for t in range(4) for h in (2, 3)}
    assert {(t, h, c) for t, h, c in bad if c != 5} == {(3, h, 9) for h in (0, 1)}
    assert bool(torch.isfinite(lse).all())
    s.close()


def test_rows_far_apart_in_the_two_parts():
    """Scores of the prefix far above or below those behind it: either part's weights may vanish."""
    for amp in (60.0, -60.0):
        s = SharedSetup([1] * 5, [80] * 5, hq=2, hk=1, dim=64, fmt="fp16", page=8).share([5], [64])
        q = torch.ones(5, 2, 64, dtype=torch.float16)
        for r in range(5):
            for side in (0,):
                s.vals[r][side] = s.vals[r][side] * 0
                s.vals[r][side][:64] = amp / 8
        s.gk.zero_()
        for p in range(64):
            s.gk[int(s.table[0, p // 8]), p % 8] = amp / 8
        out, lse = s.attend_shared(q, scale=1.0)
        check_shared(s, q, out, lse, scale=1.0)
        s.close()


# ----------------------------------------------------------------------------- streams and graphs

@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("new", [1, 40])
def test_pools_past_32_bits(fmt, new):
    """Pools of more than 2^32 elements, the used pages at both ends: attention against the oracle; what the other calls leave is
    bit for bit what they leave in a small pool."""
    page, hk, dim, prefix = 64, 8, 128, 200
    s = SharedSetup([new] * 3, [prefix + new + 50 * r for r in range(3)], hq=32, hk=hk, dim=dim, page=page, fmt=fmt, order="pch",
                    seed=new).share([3], [prefix])
    n_pages = (1 << 32) // (page * hk * dim) + 40
    small = [t for t in (s.gk, s.gv, s.gks, s.gvs) if t is not None]
    large = [torch.empty((n_pages,) + t.shape[1:], dtype=t.dtype, device="cuda") for t in small]
    where = torch.tensor([i if i % 2 else n_pages - 1 - i for i in range(s.gk.shape[0])], device="cuda")
    small_cache = s.cache
    table = torch.where(s.gtable >= 0, where[s.gtable.clamp_min(0).long()].int(), s.gtable)
    s.cache = bd.paged_cache(large[0], large[1], table, *large[2:])

    def same(move=False):
        torch.cuda.synchronize()
        for a, b in zip(small, large):
            if move:
                b[where] = a
            assert torch.equal(a.contiguous().view(torch.uint8), b[where].view(torch.uint8))

    same(move=True)
    q = s.queries("bf16")
    for how in ("together", "apart"):
        check_shared(s, q, *s.attend_shared(q, how=how))
    s.gtable[1:, :prefix // page] = s.gtable[0, :prefix // page]
    table[1:, :prefix // page] = table[0, :prefix // page]
    x = torch.randn(s.tokens, hk, dim, generator=torch.Generator().manual_seed(2)).cuda()
    copies = [[3, 0], [4, 5], [page, 7]]
    keep, n_keep = i32([[0] if new == 1 else [1, 5, 39]] * 3), i32([1 if new == 1 else 3] * 3)
    for cache, ids in ((small_cache, torch.arange(len(where), device="cuda")), (s.cache, where)):
        bd.dflash2_paged_rope_write(s.handle, bd.make_rope(dim), cache, None, None, x, x, s.begin, s.kv_len)
        bd.dflash2_paged_keep(s.handle, [cache], s.begin, s.kv_len, keep, n_keep)
        moved = torch.stack([ids[torch.tensor(c, device="cuda")].int() for c in copies[:2]] + [i32(copies[2])])
        bd.dflash2_pages_copy(s.handle, [cache], moved)
    same()
    s.close()


def test_rows_past_32_bits():
    stride = (1 << 31) + 64
    far = torch.empty(2 * stride + 256, dtype=torch.bfloat16, device="cuda").as_strided((3, 2, 64), (stride, 128, 1))
    x, plan, pos = torch.randn(3, 2, 64, device="cuda").bfloat16(), bd.make_rope(64), i32([3, 70000, 5])
    out, back = torch.empty_like(x), torch.empty_like(x)
    bd.dflash2_rope(plan, x, out, pos)
    bd.dflash2_rope(plan, x, far, pos)
    assert torch.equal(far, out)
    far.copy_(x)
    bd.dflash2_rope(plan, far, back, pos)
    assert torch.equal(back, out)


@pytest.mark.parametrize("how", ["together", "apart"])
@pytest.mark.parametrize("sizes,new", [([2] * 265, 1), ([1] * 530, 5), ([530], 1)])
def test_shared_attention_of_many_requests(sizes, new, how):
    """More groups, or more requests, than a block has threads, with host bounds far above what there is."""
    g = np.random.default_rng(len(sizes))
    prefix = (30 + g.integers(0, 90, len(sizes))).tolist()
    pre = [p for size, p in zip(sizes, prefix) for _ in range(size)]
    s = SharedSetup([new] * 530, [p + new + int(x) for p, x in zip(pre, g.integers(0, 40, 530))], hq=4, hk=1, dim=64, seed=6).share(sizes, prefix)
    s.max_group = s.tokens
    q = s.queries("bf16")
    status = torch.zeros(530, dtype=torch.int32, device="cuda")
    out, lse = s.attend_shared(q, how=how, status=status, max_prefix=1 << 20)
    assert not status.any()
    check_shared(s, q, out, lse, skip=[r for r in range(530) if r % 7 and r < 520])
    assert torch.isfinite(out.float()).all()
    s.close()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_shared_attention_of_prompts(fmt):
    """Thousands of new rows a group: prompts that go on from a common beginning."""
    s = SharedSetup([1100, 0, 515], [900 + 1100, 900, 900 + 700], hq=8, hk=1, dim=64, page=32, fmt=fmt, seed=4).share([3], [900])
    q = s.queries("bf16")
    check_shared(s, q, *s.attend_shared(q))
    s.close()


def test_captured_calls_replay_on_new_contents():
    """Two graphs with a handle and workspaces of their own, replayed in turn on lengths, tables and tokens that changed since."""
    graphs = []
    for seed in (1, 2):
        s = SharedSetup([2] * 6, [300 + 3 * r for r in range(6)], fmt="int8", page=16, seed=seed).share([4, 2], [256, 100])
        s.q = s.queries("bf16").cuda()
        s.out, s.turned = torch.zeros_like(s.q), torch.zeros_like(s.q)
        s.pages = Pages(6, 5, 40, 16)
        s.lens = i32([20] * 6)
        s.plan, s.pos = bd.make_rope(128), i32(range(12))

        def step(s=s):
            bd.dflash2_rope(s.plan, s.q, s.turned, s.pos)
            bd.dflash2_pages_resize(s.pages.pool, s.pages.kv, s.lens, s.pages.copies)
            bd.dflash2_paged_attention_shared(s.handle, s.cache, s.turned, s.out, s.begin, s.kv_len, s.group_begin, s.prefix_len, s.work,
                                              max_new=2, max_len=400, max_group=12, max_prefix=300, scale=0.1, how="together")
        step()
        torch.cuda.synchronize()
        s.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(s.graph):
            step()
        graphs.append(s)
    for turn in range(3):
        for s in graphs:
            s.pos.add_(5)
            s.kv_len.sub_(1)
            s.prefix_len[1] = 100 - turn
            s.lens.copy_(i32([20 + 16 * turn] * 6))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        for s in graphs:
            with torch.cuda.stream(side):
                s.graph.replay()
        side.synchronize()
        for s in graphs:
            assert s.pages.kv.tolist() == [20 + 16 * turn] * 6
            s.prefix, now = [256, 100 - turn], [300 + 3 * r - turn - 1 for r in range(6)]
            turned = torch.empty_like(s.q)
            bd.dflash2_rope(s.plan, s.q, turned, s.pos)
            assert torch.equal(turned, s.turned)
            out = torch.empty_like(s.out)
            bd.dflash2_paged_attention_shared(s.handle, s.cache, turned, out, s.begin, s.kv_len, s.group_begin, s.prefix_len, s.work,
                                              max_new=2, max_len=400, max_group=12, max_prefix=300, scale=0.1, how="together")
            # the same bits (the shorter second prefix uncovers rows of NaN in its second request)
            assert torch.equal(out.view(torch.int16), s.out.view(torch.int16)) and s.kv_len.tolist() == now
            assert bool(torch.isfinite(s.out[:10]).all())
    for s in graphs:
        s.close()


def test_calls_on_another_stream():
    """Work queued on a stream before a call is seen by it."""
    s = SharedSetup([1] * 8, [400] * 8, fmt="bf16").share([8], [384])
    q = s.queries("bf16").cuda()
    want, _ = s.attend_shared(q)
    side = torch.cuda.Stream()
    late, out = torch.zeros_like(q), torch.zeros_like(q)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        late.copy_(q)
    bd.dflash2_paged_attention_shared(s.handle, s.cache, late, out, s.begin, s.kv_len, s.group_begin, s.prefix_len, s.work, max_new=1,
                                      max_len=400, max_group=8, max_prefix=384, scale=s.dim ** -0.5, stream=side, how="together")
    side.synchronize()
    assert torch.equal(out, want)
    s.close()
