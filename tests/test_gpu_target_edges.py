"""Places where the target's side of a step can go wrong: what a row does not see, calls whose ranges are
partly bad, and decisions of the sampling that lie exactly on a border."""
import ctypes

import numpy as np
import pytest
import torch

import block_drafter_pos_gb300 as bd
from oracle import target as ot
from test_gpu_target import DT, HALF, MARGIN, Setup, check_attention, run_sample

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------------------- what a row does not see

@pytest.mark.parametrize("fmt", ["bf16", "fp16", "int8"])
def test_nonfinite_values_in_many_small_units(fmt):
    """Units of one and of two row tiles after one another in a CTA, nonfinite values in some of them."""
    g = np.random.default_rng(4)
    new = [int(n) for n in g.choice([20, 40], 700)]            # 80 or 160 rows per KV head
    s = Setup(new, new, hq=8, hk=2, dim=64, page=16, fmt=fmt, seed=9)
    q = s.queries("bf16" if fmt in ot.QMAX else fmt)
    clean, _ = s.attend(q)
    hit = [r for r in range(700) if g.random() < 0.3]
    for r in hit:                                              # token 10 on see it, and KV head 0 only
        (s.gv if s.gvs is None else s.gvs)[int(s.table[r, 0]), 10, 0] = float("nan")
    for _ in range(3):
        out, _ = s.attend(q)
        at = 0
        seen = torch.zeros(out.shape, dtype=torch.bool)
        for r, n in enumerate(new):
            if r in hit:
                seen[at + 10:at + n, :4] = True
            at += n
        got = out.cpu()
        assert torch.isnan(got[seen].float()).all() and torch.equal(got[~seen], clean.cpu()[~seen])
    s.close()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("n", [8, 9, 140])
@pytest.mark.parametrize("power", [14, 30, 100])
def test_a_large_value_that_a_row_does_not_see(fmt, n, power):
    """A later token's value 2^power times the others': the rows before it do not notice, nor do rows whose window has
    left it (held to bounds over what they see), and the rows that see it are right."""
    length, first = 200, 200 - n + n // 2
    s = Setup([n], [length], hq=4, hk=2, fmt=fmt, seed=n)
    q = s.queries("bf16")
    clean, lse0 = s.attend(q)
    narrow, _ = s.attend(q, window=3)
    vals = [[x.copy() for x in s.vals[0]]]                     # of the rows that do not see it
    hidden = torch.ones(n, dtype=torch.bool)
    hidden[n // 2:n // 2 + 3] = False
    s.gvs[int(s.table[0, first // 16]), first % 16, 1] *= 2.0 ** power
    s.vals[0][1][first, 1] *= 2.0 ** power
    out, lse = s.attend(q)
    assert torch.equal(out[:, :2], clean[:, :2])
    check_attention(s, q, out, lse)
    check_attention(s, q, torch.cat([out[:n // 2], clean[n // 2:]]), torch.cat([lse[:n // 2], lse0[n // 2:]]), vals=vals)
    out, _ = s.attend(q, window=3)
    assert torch.equal(out[:, :2], narrow[:, :2])
    check_attention(s, q, out, None, window=3)
    narrow[hidden] = out[hidden]
    check_attention(s, q, narrow, None, window=3, vals=vals)
    s.close()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("n", [6, 64])
def test_a_large_value_in_another_branch(fmt, n):
    """Written through the cache: a node's value 2^30 times the others' shows below it in the tree and nowhere else."""
    s = Setup([n], [n + 100], hq=4, hk=2, fmt=fmt, seed=n)
    g = np.random.default_rng(n)
    words = [1]
    for i in range(1, n):
        words.append(words[int(g.integers(0, i))] | (1 << i))
    words[1] = 3                                               # node 1 hangs on the root
    tree = np.array(words, np.uint64)
    below = torch.tensor([bool(w >> 1 & 1) for w in words])
    t = torch.from_numpy(tree.view(np.int64)).cuda()
    k, v = (torch.from_numpy(g.standard_normal((n, 2, 128)).astype(np.float32)).cuda() for _ in "kv")
    q = s.queries("bf16")
    got = []
    for factor in (2.0 ** 30, 1.0):
        v2 = v.clone()
        v2[1] *= factor
        bd.dflash2_paged_write(s.handle, s.cache, k, v2, s.begin, s.kv_len)
        got.append(s.attend(q, tree_mask=t)[0])
    for i, (x, fine) in enumerate(((k, s.vals[0][0]), (v, s.vals[0][1]))):
        codes, scale = ot.quantise(x.cpu().numpy(), fmt)
        fine[100:] = codes * scale[..., None].astype(np.float64)
    assert below.any() and not below.all() and (got[0][below].float().abs().amax((1, 2)) > 1e3).all()
    got[0][below] = got[1][below]
    for out in got:
        check_attention(s, q, out, None, tree=tree)
    s.close()


def test_rows_that_saw_a_large_value_before_a_small_one():
    """Long contexts whose scales rise and fall by 2^12 from tile to tile, windows and prompts among them."""
    for n, window in ((4, 0), (4, 300), (150, 0), (150, 300)):
        s = Setup([n, n], [900, 1300], hq=4, hk=2, dim=64, page=32, fmt="e4m3", seed=n)
        for r, length in enumerate(s.length):
            f = np.exp2(12.0 * np.sin(np.arange(length) / 90.0)).astype(np.float32)
            pos = np.arange(length)
            pages = torch.from_numpy(s.table[r][pos // 32].astype(np.int64)).cuda()
            s.gvs[pages, torch.from_numpy(pos % 32).cuda()] *= torch.from_numpy(f).cuda()[:, None]
            s.vals[r][1] *= f[:, None, None].astype(np.float64)
        q = s.queries("fp16")
        out, lse = s.attend(q, window=window)
        check_attention(s, q, out, lse, window=window)
        s.close()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("n,length,window", [(7, 40, 0), (140, 140, 0), (140, 700, 33)])
def test_value_rows_of_zeros(fmt, n, length, window):
    """Rows of zeros have the least scale, next to scales of the ordinary size and of 2^-60 of it."""
    s = Setup([n], [length], hq=4, hk=2, fmt=fmt, seed=n)
    g = np.random.default_rng(n)
    kind = g.integers(0, 3, length)
    for p in range(length):
        page, row = int(s.table[0, p // 16]), p % 16
        if kind[p] == 0:
            s.gv[page, row] = torch.zeros(2, 128).to(DT[fmt]).cuda()
            s.gvs[page, row] = 2.0 ** -126
            s.vals[0][1][p] = 0
        elif kind[p] == 1:
            s.gvs[page, row] *= 2.0 ** -60
            s.vals[0][1][p] *= 2.0 ** -60
    q = s.queries("bf16")
    for causal in (True, False):
        out, lse = s.attend(q, window=window, causal=causal)
        check_attention(s, q, out, lse, causal=causal, window=window)
    s.close()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("n,length,window", [(5, 300, 0), (140, 600, 300), (250, 250, 0), (200, 600, 0)])
@pytest.mark.parametrize("what", ["zero", "bad page"])
def test_first_tiles_without_a_scale(fmt, n, length, window, what):
    """Scales of zero, or pages outside the pool, where a unit's keys begin: the rest keeps its weight.  (Enough requests
    that a CTA has several tiles of a unit.)"""
    s = Setup([n] * 20, [length] * 20, hq=8, hk=8, dim=64, fmt=fmt, seed=n)
    q = s.queries("bf16")
    begin = max(0, length - n - window + 1) // 128 * 128 if window else 0
    for r in range(20):
        if what == "zero":
            for p in range(begin, begin + 128):
                s.gvs[int(s.table[r, p // 16]), p % 16] = 0.0
        else:
            s.gtable[r, begin // 16:begin // 16 + 8] = -1
        s.vals[r][1][begin:begin + 128] = 0
    out, lse = s.attend(q, window=window)
    see = ot.visible(n, length, True, window)
    if what != "zero":
        see[:, begin:begin + 128] = False
    for r in (0, 7, 19):
        k, v = s.vals[r]
        part = slice(r * n, (r + 1) * n)
        want, wl, spread, reach = ot.paged_attention(q.double().numpy()[part], k, v, 64 ** -0.5, see)
        tol = HALF["bf16"] * np.abs(want) + 2.0 ** -10 * spread + 2.0 ** -20 * np.abs(v).max()
        assert (np.abs(out[part].float().cpu().numpy() - want) <= tol).all()
        assert np.array_equal(np.isneginf(lse[part].cpu().numpy()), np.isneginf(wl))
    s.close()


def _dense(s, q, r, at, see, scale):
    """Request r's rows in 64 bits on the GPU: outputs, and for the bounds the weighted magnitudes, the largest visible
    value and the largest score's magnitude."""
    n = s.new[r]
    k, v = (torch.from_numpy(x).cuda() for x in s.vals[r])
    group = s.hq // s.hk
    k, v = (x.repeat_interleave(group, 1).transpose(0, 1) for x in (k, v))                    # [hq, keys, dim]
    see = torch.from_numpy(see).cuda()
    z = q[at:at + n].cuda().double().transpose(0, 1) @ k.transpose(1, 2) * scale
    reach = (q[at:at + n].cuda().double().abs().transpose(0, 1) @ k.abs().transpose(1, 2) * scale).masked_fill(~see, 0).amax(-1)
    w = torch.softmax(z.masked_fill(~see, float("-inf")), -1).nan_to_num(0.0)
    # (a position with a weight of zero adds nothing, whatever it holds; one with a weight adds what it holds)
    bad = ~torch.isfinite(v)
    out = w @ v.masked_fill(bad, 0.0)
    hit = (see.to(v.dtype)[None].expand(s.hq, -1, -1) @ bad.to(v.dtype)) > 0
    big = (see[None, :, :] & (v.masked_fill(bad, 0.0).abs().amax(-1) > 0)[:, None, :])
    top = (big * v.masked_fill(bad, 0.0).abs().amax(-1)[:, None, :]).amax(-1)
    return [x.transpose(0, 1) for x in (out, w @ v.masked_fill(bad, 0.0).abs(), hit)] + [x.T for x in (top, reach)]


@pytest.mark.parametrize("seed", range(24))
def test_spread_scales_over_many_tiles(seed):
    """Value scales that differ by up to 2^80, zeros, scales and codes that are no numbers, windows, trees, blocks and prompts,
    in runs of several tiles and units a CTA: every row against what it sees."""
    g = np.random.default_rng(seed)
    fmt = ["int8", "e4m3"][seed % 2]
    kind = ["prompt", "prompt", "block", "tree"][seed // 2 % 4]
    n_req = 24
    lo, hi = {"prompt": (20, 260), "block": (2, 8), "tree": (10, 64)}[kind]
    new = [int(x) for x in g.integers(lo, hi + 1, n_req)]
    length = [n + int(g.integers(0, 900)) for n in new]
    group = 4 if kind != "block" else int(g.choice([1, 4]))
    s = Setup(new, length, hq=4 * group, hk=4, dim=[64, 128][seed // 8 % 2], page=16, fmt=fmt, seed=seed)
    window = int(g.choice([0, 0, 40, 300]))
    causal = bool(kind != "block" or g.random() < 0.5)
    spread = float(g.choice([3, 12, 40, 80]))
    tree = None
    if kind == "tree":
        words = []
        for n in new:
            w = [1]
            for i in range(1, n):
                w.append(w[int(g.integers(0, i))] | (1 << i))
            words += w
        tree = np.array(words, np.uint64)
    for r, total in enumerate(length):
        pos = np.arange(total)
        pages, rows = torch.from_numpy(s.table[r][pos // 16].astype(np.int64)).cuda(), torch.from_numpy(pos % 16).cuda()
        # plateaus of scales, single outliers, zeros
        e = np.repeat(g.uniform(-spread / 2, spread / 2, total // 50 + 1), 50)[:total] if g.random() < 0.5 else np.zeros(total)
        e = e + np.where(g.random(total) < 0.02, g.uniform(-spread / 2, spread / 2, total), 0)
        f = np.where(g.random(total) < 0.02, 0.0, np.exp2(np.round(e)))
        s.gvs[pages, rows] *= torch.from_numpy(f.astype(np.float32)).cuda()[:, None]
        s.vals[r][1] *= f[:, None, None]
        for p in np.nonzero(g.random(total) < 0.002)[0]:           # one head of a position
            h, c = int(g.integers(0, 4)), int(g.integers(0, s.dim))
            if g.random() < 0.5 or fmt == "int8":
                s.gvs[int(s.table[r, p // 16]), p % 16, h] = float("nan")
                s.vals[r][1][p, h] = np.nan
            else:
                codes = s.gv[int(s.table[r, p // 16]), p % 16, h].view(torch.uint8).clone()
                codes[c] = 0x7F
                s.gv[int(s.table[r, p // 16]), p % 16, h] = codes.view(DT["e4m3"])
                s.vals[r][1][p, h, c] = np.nan
    q = s.queries("bf16")
    scale = s.dim ** -0.5
    out, lse = s.attend(q, window=window, causal=causal, tree_mask=None if tree is None else torch.from_numpy(tree.view(np.int64)).cuda())
    at = 0
    for r, (n, total) in enumerate(zip(new, length)):
        see = ot.visible(n, total, causal, window, None if tree is None else tree[at:at + n])
        want, sums, hit, top, reach = _dense(s, q, r, at, see, scale)
        got = out[at:at + n].double()
        # the output's rounding, one of the weights, the scores' and exponentials', and weights next to a larger scale: half of
        # fp16's least step times the reference, an 8th of the largest scale at most, for every key
        rel = 2 * reach * (s.dim * 2.0 ** -24 + 2.0 ** -23) + 2.0 ** -21 + (total / 64 + 2) * 2.0 ** -22
        tol = HALF["bf16"] * want.abs() + (HALF["fp16"] + 2 * rel[..., None]) * sums * 1.01 + total * 2.0 ** -28 * top[..., None] + 1e-30
        assert torch.equal(torch.isnan(got), hit), f"request {r}: NaN pattern"
        over = ((got - want).abs() > tol) & ~hit
        assert not over.any(), (r, kind, spread, window, (got - want).abs()[over].max().item(), tol[over].min().item())
        at += n
    s.close()


@pytest.mark.parametrize("n", [8, 140])
@pytest.mark.parametrize("byte", [0x7F, 0xFF])
@pytest.mark.parametrize("dim", [64, 128])
def test_a_code_that_is_no_number(n, byte, dim):
    """An e4m3 NaN code in a value reaches its channel in the rows that see it and nothing else; in a key, those rows."""
    length, c = 200, 37
    first = length - n + n // 2
    s = Setup([n], [length], hq=4, hk=2, dim=dim, fmt="e4m3", seed=n)
    q = s.queries("bf16")
    clean, _ = s.attend(q)
    page, row = int(s.table[0, first // 16]), first % 16
    others = [i for i in range(dim) if i != c]
    for window in (0, 5):
        base = clean if window == 0 else s.attend(q, window=window)[0]
        sees = torch.zeros(n, dtype=torch.bool)
        sees[n // 2:n if window == 0 else n // 2 + window] = True
        for pool in (s.gv, s.gk):
            keep = pool[page, row, 1].clone()
            codes = keep.view(torch.uint8).clone()
            codes[c] = byte
            pool[page, row, 1] = codes.view(DT["e4m3"])
            out, _ = s.attend(q, window=window)
            pool[page, row, 1] = keep
            assert torch.equal(out[~sees], base[~sees]) and torch.equal(out[:, :2], base[:, :2])
            late = out[sees][:, 2:]
            if pool is s.gv:
                assert torch.isnan(late[..., c].float()).all()
                assert torch.equal(late[..., others], base[sees][:, 2:][..., others])
            else:
                assert torch.isnan(late.float()).all()
    # in a position that every row sees: the channel of every row
    far = 3
    pool = s.gv[int(s.table[0, 0]), far, 1]
    codes = pool.view(torch.uint8).clone()
    codes[c] = byte
    s.gv[int(s.table[0, 0]), far, 1] = codes.view(DT["e4m3"])
    out, _ = s.attend(q)
    assert torch.isnan(out[:, 2:, c].float()).all() and torch.equal(out[:, 2:][..., others], clean[:, 2:][..., others])
    s.close()


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "bf16", "fp16"])
@pytest.mark.parametrize("qt", ["bf16", "fp16"])
@pytest.mark.parametrize("group", [1, 4, 16, 64])
def test_one_key_is_its_value(fmt, qt, group):
    """A softmax of one key weighs it 1: the output is the value, rounded once to the output's type.  (Above 32 rows per KV
    head the weight that is rounded to 16 bits and the sum may stand for a power of two next to 1: two roundings.)"""
    if fmt not in ot.QMAX and fmt != qt:
        pytest.skip("a 16-bit cache takes queries of its own type")
    s = Setup([1] * 40, [1] * 40, hq=2 * group, hk=2, fmt=fmt, seed=group, scale_spread=1e3)
    out, lse = s.attend(s.queries(qt))
    for r in range(40):
        want = torch.from_numpy(s.vals[r][1][0].astype(np.float32)).to(DT[qt])      # [heads, channels]
        got = out[r].cpu().view(2, group, 128)
        if group <= 32:
            assert torch.equal(got, want[:, None].expand(2, group, 128))
        else:
            v = torch.from_numpy(s.vals[r][1][0])[:, None]
            weight = HALF["fp16" if fmt in ot.QMAX else fmt]
            assert ((got.double() - v).abs() <= v.abs() * (HALF[qt] + weight) * 1.01 + 2.0 ** -25).all()
    s.close()


@pytest.mark.parametrize("fmt", ["bf16", "fp16", "int8", "e4m3"])
@pytest.mark.parametrize("n", [3, 8, 140])
def test_values_that_are_not_finite_under_vanishing_weights(fmt, n):
    """One-hot scores: a NaN value shows in every row that sees it, however small its weight, and in no other."""
    length = 200
    s = Setup([n], [length], hq=4, hk=2, fmt=fmt, seed=n)
    q = s.queries("bf16" if fmt in ot.QMAX else fmt, amp=60.0)
    clean, _ = s.attend(q, scale=1.0)
    for first in (length - n, length - n + n // 2, length - 1, 5):
        page, row = int(s.table[0, first // 16]), first % 16
        pool = s.gv if s.gvs is None else s.gvs
        keep = pool[page, row, 1].clone()
        pool[page, row, 1] = float("nan")
        out, _ = s.attend(q, scale=1.0)
        pool[page, row, 1] = keep
        sees = max(0, first - (length - n))
        assert torch.isnan(out[sees:, 2:].float()).all() and torch.equal(out[:sees], clean[:sees])
        assert torch.equal(out[:, :2], clean[:, :2])
    s.close()


@pytest.mark.parametrize("fmt,amp,q_amp", [("e4m3", 1.0, 2.0 ** -40), ("int8", 1.0, 2.0 ** -100), ("e4m3", 1.0, 1.0), ("bf16", 1e36, 1.0),
                                           ("fp16", 1.0, 1.0)])
@pytest.mark.parametrize("n", [5, 140])
def test_a_scale_of_zero_weighs_all_alike(fmt, amp, q_amp, n):
    s = Setup([n], [200], hq=4, hk=2, fmt=fmt, seed=n, amp=amp)
    q = s.queries("fp16" if fmt == "fp16" else "bf16", amp=q_amp)
    for scale in (0.0, -0.0):
        out, lse = s.attend(q, scale=scale)
        check_attention(s, q, out, lse, scale=0.0)
    out, lse = s.attend(q, scale=0.0, causal=False)
    check_attention(s, q, out, lse, scale=0.0, causal=False)
    for scale in (-0.05, 2.0 ** -60) if amp == 1.0 else ():
        out, lse = s.attend(q, scale=scale)
        check_attention(s, q, out, lse, scale=scale)
    s.close()


def test_a_scale_of_zero_and_queries_that_are_not_finite():
    for fmt in ("bf16", "int8"):
        for n in (5, 140):
            s = Setup([n], [200], hq=4, hk=2, fmt=fmt, seed=n)
            q = s.queries("bf16").cuda()
            clean, _ = s.attend(q, scale=0.0)
            q[2, 1, 7], q[3, 0, 9] = float("inf"), float("nan")
            out, _ = s.attend(q, scale=0.0)
            bad = torch.zeros(n, 4, dtype=torch.bool)
            bad[2, 1] = bad[3, 0] = True
            assert torch.isnan(out[bad].float()).all() and torch.equal(out[~bad], clean[~bad])
            s.close()


# ----------------------------------------------------------------------------- calls


@pytest.mark.parametrize("new,begin,tokens,length,want", [
    ([8, 0, 4], [0, 30, 8, 12], 12, [20, 20, 20], [1, 1, 0]),      # one range past the rows, one reversed
    ([4, 4, 4], [0, 4, 20, 24], 8, [20, 20, 20], [0, 1, 1]),       # two that end past the rows
    ([4, 0, 4], [0, 4, 4, 8], 8, [20, -1, 20], [0, 1, 0]),         # a bad length of a request without tokens
    ([4, 0, 4], [0, 4, 4, 8], 8, [20, 20, 33], [0, 0, 1]),         # past the page table's row
    ([4, 4, 4], [-2, 2, 6, 10], 10, [20, 20, 20], [1, 0, 0]),      # before the rows
])
def test_calls_agree_about_bad_ranges(new, begin, tokens, length, want):
    """Write, read and attention serve the same requests and flag the others."""
    s = Setup(new, [20, 20, 20], hq=4, hk=2, dim=64, fmt="int8", page=16, seed=2)
    b = torch.tensor(begin, dtype=torch.int32, device="cuda")
    n = torch.tensor(length, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(2, tokens, 2, 64, generator=g, device="cuda")
    status = torch.zeros(3, dtype=torch.int32, device="cuda")
    bd.dflash2_paged_write(s.handle, s.cache, x[0], x[1], b, n, status=status)
    assert status.tolist() == want
    status.zero_()
    y = torch.full_like(x, 7.0)
    bd.dflash2_paged_read(s.handle, s.cache, y[0], y[1], b, n, status=status)
    assert status.tolist() == want
    status.zero_()
    q = torch.randn(tokens, 4, 64, generator=g, device="cuda").bfloat16()
    out = torch.full_like(q, 7.0)
    bd.dflash2_paged_attention(s.handle, s.cache, q, out, b, n, max_new=tokens, max_len=32, scale=0.1, status=status)
    assert status.tolist() == want
    served = torch.zeros(tokens, dtype=torch.bool, device="cuda")
    for r in range(3):
        if want[r] == 0:
            served[begin[r]:begin[r + 1]] = True
    assert ((y - x).abs().amax((0, 2, 3))[served] < 0.05).all() and (y[:, ~served] == 7).all()
    assert (out[~served] == 7).all() and not (out[served] == 7).all(-1).any()
    s.close()


def test_write_with_padding_rows():
    """Rows behind the last request's (a captured call's padding) are left alone, and flag nothing."""
    s = Setup([3, 2], [20, 9], hq=2, hk=2, dim=64, fmt="fp16", page=8, seed=3)
    x = torch.randn(2, 40, 2, 64, device="cuda")
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    bd.dflash2_paged_write(s.handle, s.cache, x[0], x[1], s.begin, s.kv_len, status=status)
    y = torch.full_like(x, 7.0)
    bd.dflash2_paged_read(s.handle, s.cache, y[0], y[1], s.begin, s.kv_len, status=status)
    assert not status.any() and torch.equal(y[:, :5], x[:, :5].half().float()) and (y[:, 5:] == 7).all()
    s.close()


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("n", [1, 4, 140])
def test_pages_and_rows_in_descending_order(fmt, n):
    """Negative strides: the last page first, and a page's positions from its end."""
    b = bd.binding
    s = Setup([n], [300], hq=4, hk=2, dim=64, page=16, fmt=fmt, order="pch", seed=n)
    q = s.queries("bf16").cuda()
    want, _ = s.attend(q)
    size, quant = (1, True) if fmt == "int8" else (2, False)
    pages = s.gk.shape[0]
    k, v = s.gk.flip(0, 1).contiguous(), s.gv.flip(0, 1).contiguous()
    ks, vs = (t.flip(0, 1).contiguous() if quant else None for t in (s.gks, s.gvs))
    token, page = 2 * 64, 16 * 2 * 64
    end, send = ((pages - 1) * page + 15 * token) * size, ((pages - 1) * 32 + 15 * 2) * 4
    at = lambda t, o: None if t is None else t.data_ptr() + o  # noqa: E731
    c = b.PagedCache(at(k, end), at(v, end), at(ks, send), at(vs, send), s.gtable.data_ptr(), -page, -token, 64, -32, -2, 1,
                     s.gtable.stride(0), pages, s.gtable.shape[1])
    out = torch.full_like(q, 7.0)
    rows = lambda t: b.Rows(t.data_ptr(), t.stride(0), t.stride(1), b.T_BF16, 0)  # noqa: E731
    a = b.PagedAttentionArgs(1, n, n, 300, 1, 0, 64 ** -0.5, 0, s.begin.data_ptr(), s.kv_len.data_ptr(), rows(q), rows(out), None, None,
                             None)
    torch.cuda.synchronize()
    assert bd.lib().dflash2_paged_attention(s.handle, ctypes.byref(c), ctypes.byref(a), None) == b.OK
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    x = torch.zeros(2, n, 2, 64, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)
    bd.dflash2_paged_read(s.handle, s.cache, y[0], y[1], s.begin, s.kv_len)
    torch.cuda.synchronize()
    assert bd.lib().dflash2_paged_read(s.handle, ctypes.byref(c), 1, n, s.begin.data_ptr(), s.kv_len.data_ptr(),
                                       ctypes.byref(rows(x[0])), ctypes.byref(rows(x[1])), None, None) == b.OK
    torch.cuda.synchronize()
    assert torch.equal(x, y)
    s.close()


def test_calls_without_requests_or_rows():
    """An empty batch is no error and touches nothing."""
    s = Setup([2], [20], hq=4, hk=2, dim=64, fmt="int8", page=16)
    i32 = dict(dtype=torch.int32, device="cuda")
    none, one = torch.zeros(0, **i32), torch.zeros(1, **i32)
    x = torch.zeros(0, 2, 64, device="cuda")
    y = torch.full((3, 2, 64), 7.0, device="cuda")
    q = torch.full((3, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    for table in (s.gtable[:0], torch.zeros(0, 0, **i32)):
        cache = bd.paged_cache(s.gk, s.gv, table, s.gks, s.gvs)
        for rows, qq in ((x, q[:0]), (y, q)):
            bd.dflash2_paged_write(s.handle, cache, rows, rows, one, none)
            bd.dflash2_paged_read(s.handle, cache, rows, rows, one, none)
            bd.dflash2_paged_attention(s.handle, cache, qq, qq, one, none, max_new=0, max_len=0, scale=0.1)
            bd.dflash2_paged_attention(s.handle, cache, qq, qq, one, none, max_new=3, max_len=20, scale=0.1)
    torch.cuda.synchronize()
    assert (y == 7).all() and (q == 7).all()
    s.close()


# ----------------------------------------------------------------------------- sampling

def _in_place(x, t, k, p, m, u):
    n = x.shape[0]
    f = lambda a, d: torch.as_tensor(np.asarray(a), dtype=d).cuda()  # noqa: E731
    y = x.clone()
    token, prob = torch.full((n,), -9, dtype=torch.int32, device="cuda"), torch.full((n,), -9.0, device="cuda")
    bd.dflash2_sample(y, f(t, torch.float32), f(k, torch.int32), f(p, torch.float32), f(m, torch.float32), f(u, torch.float32),
                      token, prob=prob, kept=y)
    torch.cuda.synchronize()
    return token.cpu().numpy(), prob.cpu().numpy(), y.cpu().numpy()


@pytest.mark.parametrize("n,v", [(24, 9001), (24, 70001), (200, 40000)])
@pytest.mark.parametrize("t", [1.0, 1e6, 1e30, 3e38])
def test_kept_in_place_of_wide_rows(n, v, t):
    """Rows whose nucleus is wide: the kept logits take the logits' place, and the draw is the one of the logits."""
    g = np.random.default_rng(v)
    x = torch.from_numpy((g.standard_normal((n, v)) * 0.5).astype(np.float32)).cuda()
    x[:, ::7] = float("-inf")
    u = np.minimum(((np.arange(n) + 0.5) / n).astype(np.float32), np.float32(1 - 2.0 ** -24))
    for k, p, m in ((0, 0.6, 0.0), (0, 1.0, 0.0), (5000, 0.7, 0.0), (5000, 1.0, 0.5), (60, 0.9, 0.0)):
        args = ([t] * n, [k] * n, [p] * n, [m] * n, u)
        want = run_sample(x, *args)
        got = _in_place(x, *args)
        assert (want[3] == 0).all() and (want[2] > -1e29).sum() < x.numel()
        for a, c in zip(got, want):
            np.testing.assert_array_equal(a, c)



def _expect(x, k, p, m, u):
    """Token, probability and what stays at T = 1, for rows whose weights are 1 or (below 2^-50 of that) nothing."""
    order = np.argsort(-x, kind="stable")
    top = order[x[order] == x.max()]
    left = top[:k] if k > 0 else top
    n = len(left)
    if p < 1:
        left = left[np.arange(n) < np.float64(np.float32(p)) * n]
    left = np.sort(left)
    pick = int(np.nonzero(np.arange(1, len(left) + 1) > np.float64(np.float32(u)) * len(left))[0][0])
    return left[pick], 1.0 / len(left), left


@pytest.mark.parametrize("v", [300, 9000, 100003])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_sample_decisions_that_lie_on_a_border(v, dtype):
    """Weights that are equal to the bit: min_p = 1, u = 0 with the first ids cut, and top-p borders inside a group of
    equal logits are exact decisions, with one right answer."""
    x = np.full((8, v), -200.0, np.float32)
    x[0] = 3.0                                                 # all equal
    x[1, 1::2] = 1.0                                           # every other
    x[2, 17:] = -4.0                                           # the first ids cut
    x[3, -1] = 2.0                                             # the last alone
    x[4, [5, v // 2, v - 2]] = 0.5
    x[5, v // 3:] = float(torch.finfo(torch.bfloat16).min)     # the lowest of all, under the rest
    x[6, :100] = -1e4
    x[6, 100:] = -1e3
    x[7, 40:290] = 0.0
    xt = torch.from_numpy(x).to(DT[dtype]).cuda()
    xd = xt.float().cpu().numpy()
    for k, p, m in ((0, 1.0, 1.0), (7, 1.0, 1.0), (0, 0.5, 0.0), (0, 0.5, 1.0), (4, 0.5, 0.0), (4, 0.75, 1.0), (250, 0.5, 0.5),
                    (2000, 0.25, 0.0), (1, 0.1, 1.0), (0, 0.125, 0.25)):
        for u in (0.0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24):
            # (with top-k beyond the group of the largest, the other logits' weights are 0: they stay where only top-k cuts)
            tok, prob, kept, status = run_sample(xt, [1.0] * 8, [k] * 8, [p] * 8, [m] * 8, [u] * 8)
            assert (status == 0).all()
            for r in range(8):
                wt, wp, left = _expect(xd[r], k, p, m, u)
                assert tok[r] == wt, (r, k, p, m, u, tok[r], wt)
                assert abs(prob[r] - wp) <= wp * 2.0 ** -23
                if p < 1 or m > 0:
                    want = np.full(v, -1e30, np.float32)
                    want[left] = xd[r][left]
                    np.testing.assert_array_equal(kept[r], want, err_msg=str((r, k, p, m, u)))


def test_sample_rows_of_few_values_leave_little_undecided():
    """Rows of one, two and three values against the oracle, its two margins apart: what stays is compared wherever that
    is decided, the draw wherever both are, and few of the rows are neither."""
    v = 9000
    x = torch.zeros(10, v)
    x[1] = x[2] = torch.finfo(torch.float32).min
    x[2, 17] = 3.0
    x[3] = float("-inf")
    x[3, [5, 8999]] = 1.0
    x[4, ::2] = 1.0
    x[5] = torch.linspace(-80, 80, v)
    x[6, 4000] = 100.0
    x[7] = float("-inf")
    x[7, 8998] = -1e30
    x[8] = -1e4
    x[9] = torch.arange(v) % 3
    xd, x = x.numpy().astype(np.float64), x.cuda()
    f32 = lambda a: float(np.float32(a))  # noqa: E731
    rows = cuts = draws = 0
    for k, p, m in ((0, 1.0, 0.0), (7, 1.0, 0.0), (0, 0.5, 0.0), (4501, 0.7, 0.0), (1, 0.1, 1.0), (0, 1.0, 1.0), (v, 0.999, 1e-9)):
        for t in (1.0, 0.05, 100.0):
            for u in (0.0, 0.37, 1 - 2.0 ** -24):
                tok, prob, kept, status = run_sample(x, [t] * 10, [k] * 10, [p] * 10, [m] * 10, [u] * 10)
                assert (status == 0).all()
                for r in range(10):
                    wt, wp, stays, cut, draw = ot.truncated_sample_margins(xd[r], f32(t), k, f32(p), f32(m), f32(u))
                    rows, cuts, draws = rows + 1, cuts + (cut < MARGIN), draws + (min(cut, draw) < MARGIN)
                    if cut >= MARGIN:
                        np.testing.assert_array_equal(kept[r], np.where(stays, xd[r].astype(np.float32), np.float32(-1e30)))
                    if min(cut, draw) >= MARGIN:
                        assert tok[r] == wt and abs(prob[r] - wp) <= wp * (2.0 ** -27 + 2.0 ** -24) + 2.0 ** -43
    assert rows == 630 and cuts <= 6 and draws <= 22
