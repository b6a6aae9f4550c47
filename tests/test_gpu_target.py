"""The target's side of a step on the GPU, against the FP64 oracle: the paged cache's write and
read-back, attention of new tokens over it, and truncated sampling."""
import dataclasses

import numpy as np
import pytest
import torch

import block_drafter_pos_gb300 as bd
from oracle import target as ot

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "int8": torch.int8,
      "e4m3": torch.float8_e4m3fn}
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}   # a rounding is off by at most half a step


@dataclasses.dataclass
class Setup:
    """A pool whose unused rows and pages hold NaN (or NaN scales), and the requests' tables."""
    new: list
    length: list
    hq: int = 4
    hk: int = 2
    dim: int = 128
    page: int = 16
    fmt: str = "bf16"
    order: str = "phc"       # the pool's order of pages, positions (c) and heads: "phc" = heads outside positions
    seed: int = 0
    amp: float = 1.0
    scale_spread: float = 4.0

    def __post_init__(self):
        g = np.random.default_rng(self.seed)
        quant = self.fmt in ot.QMAX
        counts = [-(-n // self.page) for n in self.length]
        n_pages = sum(counts) + 2
        ids = g.permutation(n_pages)
        self.table = np.full((len(self.new), max(counts + [1])), -5, np.int32)     # unused entries: not a page
        at = 0
        for r, c in enumerate(counts):
            self.table[r, :c] = ids[at:at + c]
            at += c
        shape = (n_pages, self.page, self.hk, self.dim)
        self.k, self.v = (torch.full(shape, float("nan"), dtype=torch.float32) for _ in "kv")
        self.ks, self.vs = (torch.full(shape[:3], float("nan")) for _ in "kv")
        self.vals = []                                     # per request: the FP64 values [length, hk, dim]
        for r, n in enumerate(self.length):
            pair = []
            for pool, scales in ((self.k, self.ks), (self.v, self.vs)):
                x = torch.from_numpy(g.standard_normal((n, self.hk, self.dim)).astype(np.float32)) * self.amp
                pos = np.arange(n)
                pages, rows = torch.from_numpy(self.table[r][pos // self.page].astype(np.int64)), torch.from_numpy(pos % self.page)
                if quant:
                    codes = (x / self.amp * (40 if self.fmt == "int8" else 150)).clamp(-ot.QMAX[self.fmt], ot.QMAX[self.fmt])
                    codes = codes.round().to(torch.int8) if self.fmt == "int8" else codes.to(DT["e4m3"])
                    sc = torch.from_numpy(np.exp(g.uniform(0, np.log(self.scale_spread), (n, self.hk))).astype(np.float32))
                    sc = sc * self.amp * 3.0 / ot.QMAX[self.fmt]
                    pool[pages, rows] = codes.float()
                    scales[pages, rows] = sc
                    pair.append(codes.float().double().numpy() * sc.double().numpy()[..., None])
                else:
                    x = x.to(DT[self.fmt])
                    pool[pages, rows] = x.float()
                    pair.append(x.double().numpy())
            self.vals.append(pair)
        perm = {"pch": (0, 1, 2, 3), "phc": (0, 2, 1, 3), "hpc": (2, 0, 1, 3)}[self.order]
        back = np.argsort(perm)
        if quant:
            clean = [torch.nan_to_num(t, nan=0.0) for t in (self.k, self.v)]   # codes hold no NaN; the scales do
        else:
            clean = [self.k, self.v]
        self.gk, self.gv = (t.to(DT[self.fmt]).permute(*perm).contiguous().cuda().permute(*back.tolist()) for t in clean)
        p3 = perm[:3]
        b3 = np.argsort(p3)
        self.gks, self.gvs = ((t.permute(*p3).contiguous().cuda().permute(*b3.tolist()) if quant else None)
                              for t in (self.ks, self.vs))
        self.gtable = torch.from_numpy(self.table).cuda()
        self.begin = torch.tensor(np.concatenate([[0], np.cumsum(self.new)]), dtype=torch.int32).cuda()
        self.kv_len = torch.tensor(self.length, dtype=torch.int32).cuda()
        self.tokens = int(sum(self.new))
        self.cache = bd.paged_cache(self.gk, self.gv, self.gtable, self.gks, self.gvs)
        self.handle = bd.dflash2_paged_create(bd.make_paged_config(self.hq, self.hk, self.dim, self.page, self.fmt, max(8, len(self.new))))

    def queries(self, qtype, amp=1.0):
        g = np.random.default_rng(self.seed + 1)
        return (torch.from_numpy(g.standard_normal((self.tokens, self.hq, self.dim)).astype(np.float32)) * amp).to(DT[qtype])

    def attend(self, q, out=None, lse=True, scale=None, **kw):
        scale = self.dim ** -0.5 if scale is None else scale
        out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda") if out is None else out
        l = torch.full(q.shape[:2], float("nan"), device="cuda") if lse else None
        kw.setdefault("max_new", max(self.new + [1]))
        kw.setdefault("max_len", max(self.length + [1]))
        bd.dflash2_paged_attention(self.handle, self.cache, q.cuda() if not q.is_cuda else q, out, self.begin, self.kv_len,
                                   scale=scale, lse=l, **kw)
        torch.cuda.synchronize()
        return out, l

    def close(self):
        bd.dflash2_paged_destroy(self.handle)


def check_attention(s, q, out, lse, causal=True, window=0, tree=None, scale=None, skip=(), vals=None):
    """Every output against the oracle.  The bound counts the roundings: the output's own; one of the weights
    (to 16 bits, bf16 or fp16) against the sum of weighted magnitudes; the fp32 scores (D products and the fp16
    queries of an 8-bit cache: 2^-12 of a row's score at most, for rows with elements below 2^-14 of the
    largest); the exponentials (2^-22 each, and one more rescaling for every tile of 64 keys)."""
    scale = s.dim ** -0.5 if scale is None else scale
    quant = s.fmt in ot.QMAX
    qtype = {v: k for k, v in DT.items()}[q.dtype]
    half_w = HALF["fp16"] if quant or qtype == "fp16" else HALF["bf16"]
    o, l = out.float().cpu().double().numpy(), (lse.cpu().double().numpy() if lse is not None else None)
    qd = q.double().cpu().numpy()
    at = 0
    for r, (n, length) in enumerate(zip(s.new, s.length)):
        if r not in skip and n:
            see = ot.visible(n, length, causal, window, None if tree is None else tree[at:at + n])
            kk, vv = (vals or s.vals)[r]
            want, wl, spread, reach = ot.paged_attention(qd[at:at + n], kk, vv, scale, see)
            score = reach * (s.dim * 2.0 ** -24 + (2.0 ** -23))
            rel = 2 * score + 2.0 ** -21 + (length / 64 + 2) * 2.0 ** -22
            tol = HALF[qtype] * np.abs(want) + (half_w + 2 * rel[..., None]) * spread * 1.01 + 1e-30
            if quant:
                tol = tol + 2.0 ** -25 * np.abs(vv).max(initial=0)       # weights below the fp16 range of the largest
            if qtype == "fp16":
                tol = tol + 2.0 ** -25
            got = o[at:at + n]
            fine = np.isfinite(want)
            assert np.array_equal(np.isnan(got), np.isnan(want)), f"request {r}: NaN pattern"
            assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)])
            bad = np.abs(got - want)[fine] > tol[fine] if fine.any() else np.zeros(1, bool)
            assert not bad.any(), f"request {r}: {np.abs(got - want)[fine].max()} off, allowed {tol[fine][bad].min()}"
            if l is not None:
                gl = l[at:at + n]
                f = np.isfinite(wl)
                assert np.array_equal(np.isneginf(gl), np.isneginf(wl))
                ltol = rel + score + 2.0 ** -22 * (np.abs(wl) + 4)
                assert (np.abs(gl - wl)[f] <= ltol[f]).all(), f"request {r}: lse {np.abs(gl - wl)[f].max()}"
        at += n


# ----------------------------------------------------------------------------- write and read

@pytest.mark.parametrize("fmt", ["bf16", "fp16", "int8", "e4m3"])
@pytest.mark.parametrize("dim,page,src,order", [(128, 16, "bf16", "pch"), (64, 1, "fp32", "phc"), (128, 24, "fp16", "hpc"),
                                                (64, 64, "bf16", "phc")])
def test_write_then_read_is_exact(fmt, dim, page, src, order):
    """Codes, scales and values bit for bit; rows that the call does not own stay as they were."""
    new, length = [3, 0, 1, 17, 40], [3, 9, 100, 30, 41]
    s = Setup(new, length, hq=6, hk=3, dim=dim, page=page, fmt=fmt, order=order, seed=dim + page)
    g = torch.Generator().manual_seed(4)
    x = [(torch.randn(s.tokens, 3, dim, generator=g) * torch.exp(4 * torch.randn(s.tokens, 3, 1, generator=g))).to(DT[src])
         for _ in "kv"]
    if fmt in ot.QMAX:                                     # rows of zeros, NaN, an infinity, a tiny one
        x[0][5] = 0
        x[0][6, 1, 7], x[1][8, 2, dim - 1] = float("nan"), float("-inf")
        x[1][9] = x[1][9] * 0 + torch.finfo(DT[src]).tiny
    before = [t.clone() for t in (s.gk, s.gv)]
    status = torch.zeros(5, dtype=torch.int32, device="cuda")
    big = torch.zeros(2, s.tokens, 7, dim, dtype=DT[src], device="cuda")        # strided sources
    big[:, :, 2:5] = torch.stack(x).cuda()
    bd.dflash2_paged_write(s.handle, s.cache, big[0, :, 2:5], big[1, :, 2:5], s.begin, s.kv_len, status=status)
    for out in ("bf16", "fp16", "fp32"):
        wide = torch.zeros(2, s.tokens, 4, dim, dtype=DT[out], device="cuda")
        bd.dflash2_paged_read(s.handle, s.cache, wide[0, :, 1:], wide[1, :, 1:], s.begin, s.kv_len, status=status)
        torch.cuda.synchronize()
        assert not status.any() and not wide[:, :, 0].any()
        for i in range(2):
            if fmt in ot.QMAX:
                codes, scale = ot.quantise(x[i].float().numpy(), fmt)
                with np.errstate(all="ignore"):
                    want = torch.from_numpy((codes.astype(np.float32) * scale[..., None]).astype(np.float32))
            else:
                want = x[i].to(DT[fmt]).float()
            got = wide[i, :, 1:].float().cpu()
            torch.testing.assert_close(got, want.to(DT[out]).float(), rtol=0, atol=0, equal_nan=True)
    touched = torch.zeros(s.gk.shape[:2], dtype=torch.bool)
    for r in range(5):
        for p in range(length[r] - new[r], length[r]):
            touched[s.table[r, p // page], p % page] = True
    for pool, old in zip((s.gk, s.gv), before):
        a, c = (t.contiguous().view(torch.uint8).cpu().view(*t.shape[:3], -1) for t in (pool, old))
        assert torch.equal(a[~touched], c[~touched])
    s.close()


def test_write_and_read_flag_bad_requests():
    """Bad lengths, ranges and page ids touch nothing, and the other requests are served."""
    s = Setup([4, 4, 4, 4], [20, 20, 20, 20], fmt="int8", page=16)
    s.gtable[1, 1] = s.gk.shape[0]                         # past the pool
    s.kv_len[2] = 2                                        # fewer positions than new tokens
    s.kv_len[3] = 2 * 16 + 1                               # past the page table's row
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(16, 2, 128, generator=g, device="cuda", dtype=torch.bfloat16)
    before = (s.gk.clone(), s.gks.clone())
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    bd.dflash2_paged_write(s.handle, s.cache, x, x, s.begin, s.kv_len, status=status)
    assert status.tolist() == [0, 1, 1, 1]
    rows = torch.ones(s.gk.shape[:2], dtype=torch.bool, device="cuda")
    rows[int(s.table[0, 1]), 0:4] = False                  # request 0: positions 16 .. 19
    assert torch.equal(s.gk[rows], before[0][rows]) and not torch.equal(s.gk[~rows], before[0][~rows])
    status.zero_()
    out = torch.full((2, 16, 2, 128), 7.0, device="cuda")
    bd.dflash2_paged_read(s.handle, s.cache, out[0], out[1], s.begin, s.kv_len, status=status)
    assert status.tolist() == [0, 1, 1, 1]
    assert (out[:, 4:8] == 0).all() and (out[:, 8:] == 7).all()     # a bad page reads zeros, a bad request nothing
    assert (out[0, :4] - x[:4].float()).abs().max() < 0.05
    s.close()


# ----------------------------------------------------------------------------- attention

FORMATS = [("bf16", "bf16"), ("fp16", "fp16"), ("int8", "bf16"), ("int8", "fp16"), ("e4m3", "bf16"), ("e4m3", "fp16")]


@pytest.mark.parametrize("fmt,qt", FORMATS)
@pytest.mark.parametrize("dim", [128, 64])
@pytest.mark.parametrize("new,length,hq,hk,page", [
    ([1], [1], 1, 1, 16),                                  # one token, itself only
    ([1, 1, 1], [63, 64, 65], 8, 2, 16),                   # tile borders
    ([1] * 5, [2, 700, 129, 1, 1000], 12, 2, 24),          # ragged decoding, odd group and page
    ([8, 8], [300, 8], 8, 2, 32),                          # verify blocks, one with no context
    ([2, 7, 3], [90, 77, 500], 4, 4, 1),                   # no sharing, pages of one position
    ([5, 0, 16, 1], [70, 10, 400, 333], 8, 1, 48),         # a request without new tokens
    ([40], [131], 6, 2, 64),                               # more rows than one unit holds
    ([70, 33], [70, 200], 4, 2, 16),                       # prompts
    ([1, 3], [140, 9], 64, 1, 16),                         # the widest group
])
def test_attention_causal(fmt, qt, dim, new, length, hq, hk, page):
    s = Setup(new, length, hq=hq, hk=hk, dim=dim, page=page, fmt=fmt, seed=len(new) + page)
    q = s.queries(qt)
    out, lse = s.attend(q)
    check_attention(s, q, out, lse)
    again, lse2 = s.attend(q)
    assert torch.equal(out, again) and torch.equal(lse, lse2)       # bit-equal when run again
    s.close()


@pytest.mark.parametrize("fmt,qt", [("bf16", "bf16"), ("e4m3", "bf16"), ("int8", "fp16")])
@pytest.mark.parametrize("new,length,window,causal", [
    ([1, 1], [100, 500], 64, True), ([8, 8, 3], [400, 9, 50], 17, True), ([70, 140], [300, 150], 33, True),
    ([4], [260], 1, True), ([8, 5], [200, 5], 100, False), ([16, 130], [16, 300], 0, False), ([6], [300], 2048, True),
    ([4], [260], 2147483647, True),
])
def test_attention_windows_and_blocks(fmt, qt, new, length, window, causal):
    s = Setup(new, length, hq=8, hk=2, page=24, fmt=fmt, seed=window % 97)
    q = s.queries(qt)
    out, lse = s.attend(q, window=window, causal=causal)
    check_attention(s, q, out, lse, causal=causal, window=window)
    s.close()


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("n,length,group", [(1, 30, 4), (9, 9, 2), (33, 200, 4), (64, 130, 3)])
def test_attention_tree(fmt, n, length, group):
    s = Setup([n, n], [length, length + 13], hq=2 * group, hk=2, fmt=fmt, page=16, seed=n)
    g = np.random.default_rng(n)
    words = []
    for r in range(2):
        w = [1]
        for i in range(1, n):
            w.append(w[int(g.integers(0, i))] | (1 << i))
        words += w
    tree = np.array(words, np.uint64)
    q = s.queries("bf16")
    t = torch.from_numpy(tree.view(np.int64)).cuda()
    out, lse = s.attend(q, tree_mask=t)
    check_attention(s, q, out, lse, tree=tree)
    out, lse = s.attend(q, tree_mask=t, window=20)
    check_attention(s, q, out, lse, tree=tree, window=20)
    s.close()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [4, 40])
def test_rows_that_see_nothing_are_zero(fmt, n):
    """Empty tree words without a context, an empty cache, and positions before the cache's start."""
    s = Setup([n, n, n], [n, 0, 2], hq=8, hk=2, fmt=fmt)
    q = s.queries("bf16")
    tree = np.zeros(3 * n, np.uint64)
    tree[1] = 2                                            # request 0: token 1 sees itself
    tree[2 * n:] = 1                                       # (a length of 2: bit 0 is position 2 - n)
    out, lse = s.attend(q, tree_mask=torch.from_numpy(tree.view(np.int64)).cuda())
    check_attention(s, q, out, lse, tree=tree)
    assert not out[0].any() and out[1].any() and torch.isneginf(lse[2]).all()
    out, lse = s.attend(q)
    check_attention(s, q, out, lse)
    assert not out[n:2 * n].any()
    s.close()


@pytest.mark.parametrize("fmt", ["bf16", "fp16", "int8", "e4m3"])
@pytest.mark.parametrize("n", [8, 140])
def test_nonfinite_values_in_masked_places_carry_nothing(fmt, n):
    """A later token's key or value that is not finite shows in the rows that see it, and in no other."""
    length = 200
    s = Setup([n], [length], hq=4, hk=2, fmt=fmt, seed=n)
    q = s.queries("bf16" if fmt in ot.QMAX else fmt)
    clean, _ = s.attend(q)
    first = length - n + n // 2                            # tokens from n // 2 on see it
    page, row = int(s.table[0, first // 16]), first % 16
    for pool, scales, value in ((s.gv, s.gvs, float("inf")), (s.gv, s.gvs, float("nan")), (s.gk, s.gks, float("nan"))):
        keep = (pool if scales is None else scales)[page, row, 1].clone()
        (pool if scales is None else scales)[page, row, 1] = value
        out, _ = s.attend(q)
        assert torch.equal(out[:n // 2], clean[:n // 2]) and torch.equal(out[:, :2], clean[:, :2])
        seen = out[n // 2:, 2:].float()
        assert not torch.isfinite(seen).any()
        win, _ = s.attend(q, window=5)                     # and past the window again
        late = slice(n // 2 + 5, n)
        assert torch.isfinite(win[late].float()).all() and torch.isfinite(win[:n // 2].float()).all()
        (pool if scales is None else scales)[page, row, 1] = keep
    s.close()


def test_infinite_scores_and_extreme_inputs():
    s = Setup([3], [70], hq=2, hk=1, fmt="bf16", amp=1.0)
    q = s.queries("bf16", amp=200.0)                       # scores of thousands: a one-hot softmax
    out, lse = s.attend(q)
    check_attention(s, q, out, lse)
    out, lse = s.attend(q, scale=-0.3)
    check_attention(s, q, out, lse, scale=-0.3)
    out, lse = s.attend(q, scale=0.0)                      # the mean of the values
    check_attention(s, q, out, lse, scale=0.0)
    s.close()
    s = Setup([3], [70], hq=2, hk=1, fmt="int8", amp=1e-30, scale_spread=1e4)   # tiny values, spread scales
    q = s.queries("bf16", amp=3e34)
    out, lse = s.attend(q)
    check_attention(s, q, out, lse)
    s.close()


def test_attention_strided_rows_and_orders():
    """Queries inside a fused projection's rows, heads outside tokens, every order of the pool."""
    for order in ("pch", "phc", "hpc"):
        for fmt in ("bf16", "e4m3"):
            s = Setup([9, 3], [90, 33], hq=8, hk=2, fmt=fmt, page=24, order=order, seed=3)
            q = s.queries("bf16")
            fused = torch.full((s.tokens, 12, s.dim), float("nan"), dtype=torch.bfloat16, device="cuda")
            fused[:, :8] = q.cuda()
            out = torch.full((8, s.tokens, s.dim), float("nan"), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
            got, lse = s.attend(fused[:, :8], out=out)
            check_attention(s, q, got, lse)
            s.close()


def test_attention_flags_bad_requests_and_pages():
    s = Setup([4, 4, 4, 4], [40, 40, 40, 40], hq=4, hk=2, fmt="bf16")
    q = s.queries("bf16").cuda()
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    good, _ = s.attend(q, status=status)
    assert not status.any()
    s.kv_len[1] = 49                                       # past the table's row (3 pages of 16)
    s.gtable[2, 0] = -1
    s.kv_len[3] = 41                                       # past the bound that the caller gave
    out, lse = s.attend(q, status=status, max_len=40)
    assert status.tolist() == [0, 1, 1, 1]
    assert torch.equal(out[:4], good[:4])
    assert torch.isnan(out[4:8].float()).all() and torch.isnan(out[12:].float()).all()   # rows left as they were
    vals = [[x[16:] for x in p] for p in s.vals]           # request 2: positions 0 .. 15 masked
    s2 = dataclasses.replace(s)                            # (same numbers; only the lengths are used below)
    s2.new, s2.length = [0, 0, 4, 0], [0, 0, 24, 0]
    o2 = out[8:12]
    check_attention(s2, q[8:12].cpu(), o2, None, vals=vals)
    s.close()


def test_attention_on_a_side_stream_and_in_a_graph():
    """Runs on the caller's stream; a captured call replays on new contents."""
    s = Setup([8] * 4, [500, 100, 64, 1000], hq=32, hk=8, fmt="bf16", seed=2)
    q = s.queries("bf16")
    qd = torch.zeros(q.shape, dtype=q.dtype, device="cuda")
    out = torch.zeros_like(qd)
    lse = torch.zeros(q.shape[:2], device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(20):
            qd.mul_(1.0)
        qd.copy_(q)
        s.attend(qd, out=out)
    side.synchronize()
    check_attention(s, q, out, None)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bd.dflash2_paged_attention(s.handle, s.cache, qd, out, s.begin, s.kv_len, max_new=8, max_len=1000,
                                   scale=s.dim ** -0.5, lse=lse)
    q2 = q.flip(0)
    qd.copy_(q2)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    check_attention(s, q2, out, lse)
    s.close()


@pytest.mark.parametrize("n", [1, 200])
def test_offsets_past_32_bits(n):
    """A pool of more than 2^32 elements, its used pages at both ends."""
    page, hk, dim = 64, 8, 128
    n_pages = (1 << 32) // (page * hk * dim) + 10
    k = torch.empty(n_pages, page, hk, dim, dtype=torch.int8, device="cuda")
    v = torch.empty_like(k)
    ks, vs = (torch.empty(n_pages, page, hk, device="cuda") for _ in "kv")
    s = Setup([n], [320], hq=8, hk=8, dim=128, page=64, fmt="int8", seed=8)
    where = [n_pages - 1, 0, n_pages - 7, 5, n_pages - 2]
    for i, p in enumerate(where):
        src = int(s.table[0, i])
        k[p], v[p], ks[p], vs[p] = s.gk[src], s.gv[src], s.gks[src], s.gvs[src]
    s.gtable[0, :5] = torch.tensor(where, dtype=torch.int32)
    s.cache = bd.paged_cache(k, v, s.gtable, ks, vs)
    q = s.queries("bf16")
    out, lse = s.attend(q)
    check_attention(s, q, out, lse)
    x = torch.randn(n, 8, 128, device="cuda")
    y = torch.empty(2, n, 8, 128, device="cuda")
    bd.dflash2_paged_write(s.handle, s.cache, x, x, s.begin, s.kv_len)
    bd.dflash2_paged_read(s.handle, s.cache, y[0], y[1], s.begin, s.kv_len)
    codes, scale = ot.quantise(x.cpu().numpy(), "int8")
    want = torch.from_numpy((codes.astype(np.float32) * scale[..., None]).astype(np.float32))
    assert torch.equal(y[0].cpu(), want) and torch.equal(y[1].cpu(), want)
    s.close()


@pytest.mark.parametrize("fmt,qt,dim", [("bf16", "bf16", 128), ("fp16", "fp16", 64), ("e4m3", "bf16", 128), ("int8", "fp16", 64)])
def test_attention_long_and_mixed(fmt, qt, dim):
    """A long context split over many CTAs next to short ones, prompts next to single tokens."""
    s = Setup([1, 150, 1, 20], [9000, 700, 3, 2500], hq=4, hk=2, dim=dim, page=32, fmt=fmt, seed=12)
    q = s.queries(qt)
    out, lse = s.attend(q)
    check_attention(s, q, out, lse)
    out, lse = s.attend(q, window=700, max_len=20000)
    check_attention(s, q, out, lse, window=700)
    s.close()


@pytest.mark.parametrize("n,group", [(1, 4), (5, 8)])
def test_attention_of_many_requests(n, group):
    """More requests than a block has threads, most of them short."""
    g = np.random.default_rng(n)
    length = (n + g.integers(0, 40, 530)).tolist()
    s = Setup([n] * 530, length, hq=group, hk=1, dim=64, fmt="bf16", seed=5)
    q = s.queries("bf16")
    out, lse = s.attend(q)
    check_attention(s, q, out, lse, skip=[r for r in range(530) if r % 7 and r < 520])
    assert torch.isfinite(out.float()).all()
    s.close()


# ----------------------------------------------------------------------------- sampling

def run_sample(x, t, k, p, m, u, kept=True):
    n, v = x.shape
    dev = "cuda"
    f = lambda a, d: None if a is None else torch.as_tensor(np.asarray(a), dtype=d).to(dev)  # noqa: E731
    token = torch.full((n,), -9, dtype=torch.int32, device=dev)
    prob = torch.full((n,), -9.0, device=dev)
    status = torch.full((n,), -9, dtype=torch.int32, device=dev)
    ko = torch.full((n, v), 5.0, device=dev) if kept else None
    bd.dflash2_sample(x, f(t, torch.float32), f(k, torch.int32), f(p, torch.float32), f(m, torch.float32),
                      f(u, torch.float32), token, prob=prob, kept=ko, status=status)
    torch.cuda.synchronize()
    return token.cpu().numpy(), prob.cpu().numpy(), None if ko is None else ko.cpu().numpy(), status.cpu().numpy()


# weights carry 29 bits with errors of either sign, and sums of them are exact: a decision further than this from
# its border is certain (probabilities: 2^-29 for the token's weight, and as much for the sum, and the fp32 result)
MARGIN = 2.0 ** -27


def check_sample(x, t, k, p, m, u):
    tok, prob, kept, status = run_sample(x, t, k, p, m, u)
    xd = x.float().cpu().numpy().astype(np.float64)
    undecided = 0
    f32 = lambda a, i: float(np.float32(a[i]))  # noqa: E731
    for r in range(len(xd)):
        wt, wp, stays, margin = ot.truncated_sample(xd[r], f32(t, r), int(k[r]), f32(p, r), f32(m, r), f32(u, r))
        assert status[r] == 0
        if margin < MARGIN:
            undecided += 1
            continue
        assert tok[r] == wt, (r, tok[r], wt, margin)
        assert abs(prob[r] - wp) <= wp * (2.0 ** -27 + 2.0 ** -24) + 2.0 ** -43
        np.testing.assert_array_equal(kept[r], np.where(stays, xd[r].astype(np.float32), np.float32(-1e30)))
    return undecided


@pytest.mark.parametrize("v", [1, 2, 31, 1000, 8192, 8193, 50001, 248320])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_sample_against_the_oracle(v, dtype):
    """bf16 rows are full of equal logits: the thresholds fall inside groups of them."""
    n = 12 if v > 10000 else 40
    g = np.random.default_rng(v)
    x = torch.from_numpy(g.standard_normal((n, v)) * g.uniform(0.3, 4, (n, 1))).to(DT[dtype]).cuda()
    t = g.uniform(0.3, 1.5, n)
    t[::7] = 0
    k = np.where(g.random(n) < 0.4, 0, g.integers(1, 300, n))
    p = np.where(g.random(n) < 0.3, 1.0, g.uniform(0.05, 0.999, n))
    m = np.where(g.random(n) < 0.5, 0.0, g.uniform(0, 0.3, n))
    u = g.random(n).astype(np.float32)
    u = np.minimum(u, np.float32(1 - 2.0 ** -24))
    u[1] = 0.0
    assert check_sample(x, t, k, p, m, u) <= n // 10


def mixed_rows(n, v, wide, seed):
    """Settings and logits of n rows, a share `wide` of them top-p without top-k."""
    g = np.random.default_rng(seed)
    x = torch.from_numpy((g.standard_normal((n, v)) * g.uniform(0.3, 3, (n, 1))).astype(np.float32)).cuda()
    long = g.random(n) < wide
    t = np.where(g.random(n) < 0.1, 0.0, g.uniform(0.5, 1.3, n))
    k = np.where(long, 0, g.integers(1, 200, n))
    p = np.where(long, g.uniform(0.3, 0.95, n), np.where(g.random(n) < 0.5, 1.0, 0.9))
    m = np.where(g.random(n) < 0.5, 0.0, g.uniform(0, 0.1, n))
    return x, t, k, p, m, np.minimum(g.random(n).astype(np.float32), np.float32(1 - 2.0 ** -24))


@pytest.mark.parametrize("n,v", [(30, 140001), (128, 33000), (600, 17001)])
@pytest.mark.parametrize("wide", [0.0, 0.05, 0.6, 1.0])
def test_sample_many_rows(n, v, wide):
    """Rows of a wide nucleus, none to all, among others that are not; more rows than a block has threads."""
    assert check_sample(*mixed_rows(n, v, wide, n)) <= n // 10


@pytest.mark.parametrize("wide", [0.1, 0.9])
def test_sample_many_rows_in_a_graph(wide):
    """What follows on the stream, eager or captured, sees every row's result."""
    x, t, k, p, m, u = mixed_rows(128, 40000, wide, 3)
    want = run_sample(x, t, k, p, m, u)
    f = [torch.as_tensor(np.asarray(a), dtype=torch.float32).cuda() for a in (t, p, m, u)]
    kk = torch.as_tensor(k, dtype=torch.int32).cuda()
    token = torch.zeros(128, dtype=torch.int32, device="cuda")
    kept = torch.zeros_like(x)

    def step():
        token.fill_(-9)
        kept.fill_(5.0)
        bd.dflash2_sample(x, f[0], kk, f[1], f[2], f[3], token, kept=kept)
        return token.clone(), kept.clone()

    eager = [step() for _ in range(10)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for got in eager:
        assert (got[0].cpu().numpy() == want[0]).all() and (got[1].cpu().numpy() == want[2]).all()
    for _ in range(3):
        out[0].zero_()
        graph.replay()
        assert (out[0].cpu().numpy() == want[0]).all() and (out[1].cpu().numpy() == want[2]).all()


def test_sample_equal_logits_and_borders():
    """Rows of one value, two values, the type's lowest value, -infinity, and single tokens left."""
    v = 9000
    low = torch.finfo(torch.float32).min
    x = torch.zeros(10, v)
    x[1] = low
    x[2] = low
    x[2, 17] = 3.0
    x[3] = float("-inf")
    x[3, [5, 8999]] = torch.tensor([1.0, 1.0])
    x[4, ::2] = 1.0
    x[5] = torch.linspace(-80, 80, v)
    x[6, 4000] = 100.0
    x[7] = float("-inf")
    x[7, 8998] = -1e30
    x[8] = -1e4
    x[9] = torch.arange(v) % 3
    x = x.cuda()
    for k, p, m in [(0, 1.0, 0.0), (7, 1.0, 0.0), (0, 0.5, 0.0), (4501, 0.7, 0.0), (1, 0.1, 1.0), (0, 1.0, 1.0), (v, 0.999, 1e-9)]:
        for t in (1.0, 0.05, 100.0):
            for u in (0.0, 0.37, 1 - 2.0 ** -24):
                check_sample(x, [t] * 10, [k] * 10, [p] * 10, [m] * 10, [u] * 10)


def test_sample_options_off_and_greedy():
    g = np.random.default_rng(2)
    x = torch.from_numpy(g.standard_normal((6, 3000))).to(torch.float16).cuda()
    x[2, 100] = x[2, 2900] = 9.0                           # greedy: the smaller id
    tok, prob, kept, status = run_sample(x, [0.0] * 6, None, None, None, [0.5] * 6)
    xd = x.float().cpu().numpy()
    assert (status == 0).all() and (prob == 1).all()
    for r in range(6):
        assert tok[r] == int(np.argmax(xd[r]))
        assert (kept[r] > -1e29).sum() == 1 and kept[r, tok[r]] == xd[r, tok[r]]
    a = run_sample(x, [0.8] * 6, None, None, None, [0.5] * 6, kept=False)
    c = run_sample(x, [0.8] * 6, [0] * 6, [1.0] * 6, [0.0] * 6, [0.5] * 6)
    assert (a[0] == c[0]).all() and (a[1] == c[1]).all()


def test_sample_flags_bad_rows():
    x = torch.zeros(12, 9000)
    x[0, 4] = float("nan")
    x[1, 8999] = float("inf")
    x[2] = float("-inf")
    t, k, p, m, u = [1.0] * 12, [5] * 12, [0.9] * 12, [0.1] * 12, [0.5] * 12
    t[3], t[4], t[5] = -1.0, float("nan"), float("inf")
    p[6], p[7] = 0.0, float("nan")
    m[8], m[9] = -0.1, 1.5
    u[10] = 1.0
    tok, prob, kept, status = run_sample(x.cuda(), t, k, p, m, u)
    assert status.tolist() == [2, 2, 2, 1, 1, 1, 1, 1, 1, 1, 1, 0]
    assert (tok[:11] == -1).all() and (prob[:11] == 0).all() and (kept[:11] == np.float32(-1e30)).all()
    assert tok[11] == 2 and abs(prob[11] - 0.2) < 1e-7     # 5 equal ids stay, the middle of them


def test_sample_strided_rows_in_place_and_another_stream():
    g = np.random.default_rng(6)
    store = torch.from_numpy(g.standard_normal((5, 12000)).astype(np.float32)).cuda()
    x = store[:, :9001]
    t, k, p, m, u = [0.7] * 5, [50] * 5, [0.9] * 5, [0.01] * 5, [0.1, 0.3, 0.5, 0.7, 0.9]
    assert check_sample(x, t, k, p, m, u) == 0
    want = run_sample(x, t, k, p, m, u)
    tail = store[:, 9001:].clone()
    side = torch.cuda.Stream()
    token = torch.zeros(5, dtype=torch.int32, device="cuda")
    f = [torch.tensor(a, device="cuda") for a in (t, p, m, u)]
    kk = torch.tensor(k, dtype=torch.int32, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        bd.dflash2_sample(x, f[0], kk, f[1], f[2], f[3], token, kept=x)
    side.synchronize()
    assert (token.cpu().numpy() == want[0]).all() and (x.cpu().numpy() == want[2]).all() and torch.equal(store[:, 9001:], tail)


def test_sample_draws_follow_the_distribution():
    """4096 rows of one distribution and evenly spread uniforms: the counts are the probabilities."""
    n = 4096
    g = np.random.default_rng(0)
    row = torch.from_numpy(g.standard_normal(600).astype(np.float32)) * 2
    x = row.repeat(n, 1).cuda()
    u = (np.arange(n) + 0.5) / n
    tok, prob, _, _ = run_sample(x, [0.9] * n, [40] * n, [0.95] * n, [0.01] * n, u, kept=False)
    _, _, stays, _ = ot.truncated_sample(row.numpy(), float(np.float32(0.9)), 40, float(np.float32(0.95)), float(np.float32(0.01)), 0.5)
    w = np.where(stays, np.exp(row.numpy().astype(np.float64) / 0.9), 0)
    w /= w.sum()
    assert np.abs(np.bincount(tok, minlength=600) / n - w).max() <= 1.01 / n
    assert np.abs(prob - w[tok]).max() < 1e-6
