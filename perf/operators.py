"""The target's side of a draft + verify step, as it is measured: writing the new tokens' keys and
values into a paged cache (quantised as they are written) and reading a range of it back, attention
of new tokens over that cache, and truncated sampling from given uniforms.

`run` computes each operator in elementary torch operations (32 bits; the sampling, whose decisions
sit next to borders, in 64), or, with `own`, through the package's entry points.
"""
import functools

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "int8": torch.int8,
      "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "int8": 1, "e4m3": 1}
QMAX = {"int8": 127.0, "e4m3": 448.0}
VOCAB = 248320           # the full drafter geometry's vocabulary


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # the K/V of one verify block (anchor + 7 proposals) of one request: launch latency
        {"name": "append_block", "op": "append", "n_req": 1, "chunk": 8, "ragged": 0.0, "ctx": 1024, "n_kv": 8, "dim": 128,
         "page": 16, "fmt": "int8", "src": "bf16", "out": "bf16"},
        # the K/V of five prompts' chunks, of unequal lengths, quantised to 8-bit floats
        {"name": "append_prompts", "op": "append", "n_req": 5, "chunk": 8001, "ragged": 0.7, "ctx": 12000, "n_kv": 8,
         "dim": 128, "page": 64, "fmt": "e4m3", "src": "bf16", "out": "bf16"},
        # one short range of a toy-sized cache (a window kept by a host-side tool)
        {"name": "read_range", "op": "read", "n_req": 1, "chunk": 77, "ragged": 0.0, "ctx": 300, "n_kv": 1, "dim": 128, "page": 8,
         "fmt": "fp16", "out": "fp32"},
        # the 2048-key windows of 16 requests, read back for the drafter's contiguous bf16 caches
        {"name": "read_windows", "op": "read", "n_req": 16, "chunk": 2047, "ragged": 0.0, "ctx": 8192, "n_kv": 8, "dim": 128,
         "page": 64, "fmt": "int8", "out": "bf16"},
        # plain decoding, one request, one token
        {"name": "token_1", "op": "attn", "n_req": 1, "chunk": 1, "ragged": 0.0, "ctx": 1024, "n_q": 32, "n_kv": 8, "dim": 128,
         "page": 16, "fmt": "bf16", "q": "bf16", "window": 0, "tree": False, "lse": False},
        # plain decoding of a full batch with ragged contexts over an 8-bit cache
        {"name": "tokens_64", "op": "attn", "n_req": 64, "chunk": 1, "ragged": 0.8, "ctx": 16384, "n_q": 32, "n_kv": 8,
         "dim": 128, "page": 16, "fmt": "e4m3", "q": "bf16", "window": 0, "tree": False, "lse": True},
        # the verify blocks (anchor + 7 proposals) of 16 requests over an int8 cache
        {"name": "blocks_16", "op": "attn", "n_req": 16, "chunk": 8, "ragged": 0.5, "ctx": 8192, "n_q": 32, "n_kv": 8,
         "dim": 128, "page": 32, "fmt": "int8", "q": "bf16", "window": 0, "tree": False, "lse": False},
        # draft trees of 32 nodes and their root, four requests, a window of 2048 keys, pages of an odd size
        {"name": "trees_4", "op": "attn", "n_req": 4, "chunk": 33, "ragged": 0.0, "ctx": 4099, "n_q": 32, "n_kv": 8,
         "dim": 128, "page": 24, "fmt": "bf16", "q": "bf16", "window": 2048, "tree": True, "lse": True},
        # several prompts' chunks at once: ragged, odd, windowed, 8-bit cache, heads of 64
        {"name": "chunk_ragged", "op": "attn", "n_req": 5, "chunk": 1501, "ragged": 0.9, "ctx": 9001, "n_q": 24, "n_kv": 4,
         "dim": 64, "page": 48, "fmt": "e4m3", "q": "fp16", "window": 2048, "tree": False, "lse": True},
        # one long prompt's last chunk: the largest
        {"name": "chunk_prompt", "op": "attn", "n_req": 1, "chunk": 4096, "ragged": 0.0, "ctx": 32768, "n_q": 32, "n_kv": 8,
         "dim": 128, "page": 64, "fmt": "bf16", "q": "bf16", "window": 0, "tree": False, "lse": False},
        # one row at the full vocabulary: the anchor after a prompt
        {"name": "sample_1", "op": "sample", "rows": 1, "vocab": VOCAB, "dtype": "fp32", "kept": False, "greedy": False},
        # all target rows of 16 requests' blocks, mixed settings, with the truncated rows for the verify
        {"name": "sample_128", "op": "sample", "rows": 128, "vocab": VOCAB, "dtype": "fp32", "kept": True, "greedy": True},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["append", "read", "attn", "attn", "sample"])
    page = rng.choice([1, 8, 16, 24, 32, 48, 64, 128])
    fmt = rng.choice(["bf16", "fp16", "int8", "e4m3"])
    n_kv, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    if op in ("append", "read"):
        chunk = _log_int(rng, 1, 8000)
        c = {"op": op, "n_req": _log_int(rng, 1, 5 if op == "append" else 16), "chunk": chunk,
             "ragged": round(rng.random() * 0.9, 2), "ctx": chunk + _log_int(rng, 1, 4000), "n_kv": n_kv, "dim": dim,
             "page": page, "fmt": fmt, "out": rng.choice(["bf16", "fp16", "fp32"])}
        if op == "append":
            c["src"] = rng.choice(["bf16", "fp16", "fp32"])
        return c
    if op == "sample":
        return {"op": op, "rows": _log_int(rng, 1, 128), "vocab": _log_int(rng, 1000, VOCAB),
                "dtype": rng.choice(["fp32", "bf16", "fp16"]), "kept": rng.random() < 0.5, "greedy": rng.random() < 0.5}
    kind = rng.choice(["token", "block", "tree", "chunk"])
    group = rng.choice([1, 2, 3, 4, 6, 8])
    if kind == "token":
        n_req, chunk, ctx = _log_int(rng, 1, 64), 1, _log_int(rng, 1, 16384)
    elif kind == "block":
        n_req, chunk, ctx = _log_int(rng, 1, 16), rng.randint(2, 16), _log_int(rng, 17, 8192)
    elif kind == "tree":
        n_req, chunk, ctx = _log_int(rng, 1, 16), rng.randint(2, 64), _log_int(rng, 70, 4100)
    else:
        n_req, chunk = _log_int(rng, 1, 8), _log_int(rng, 65, 2048)
        ctx = chunk + _log_int(rng, 1, 14000)
    # no drawn case costs more than the largest listed one: heads * queries * keys
    ctx = max(chunk, min(ctx, 4096 * 32768 * 32 // (n_req * chunk * n_kv * group)))
    return {"op": op, "n_req": n_req, "chunk": chunk, "ragged": round(rng.random() * 0.9, 2), "ctx": ctx,
            "n_q": n_kv * group, "n_kv": n_kv, "dim": dim, "page": page, "fmt": fmt,
            "q": fmt if fmt in ("bf16", "fp16") else rng.choice(["bf16", "fp16"]),
            "window": rng.choice([0, 0, 2048, rng.randint(1, 4000)]), "tree": kind == "tree", "lse": rng.random() < 0.5}


def _lengths(case):
    """New tokens and cache lengths (new tokens included) of each request: the first request's are the
    case's, the others' fall by up to the share `ragged`, and keep at least one new token."""
    n = case["n_req"]
    cut = [case["ragged"] * ((r * 5) % n) / n for r in range(n)]
    new = [max(1, int(case["chunk"] * (1 - c))) for c in cut]
    return new, [max(m, int(case["ctx"] * (1 - c))) for m, c in zip(new, cut)]


# ------------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    if case["op"] == "sample":
        return _prepare_sample(case, g, dev)
    new, total = _lengths(case)
    page, n_kv, dim, fmt = case["page"], case["n_kv"], case["dim"], case["fmt"]
    counts = [-(-t // page) for t in total]
    n_pages = sum(counts) + 3
    ids = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)  # pages in no order, as a pool's
    table = torch.zeros(case["n_req"], max(counts), dtype=torch.int32, device=dev)
    at = 0
    for r, c in enumerate(counts):
        table[r, :c] = ids[at:at + c]
        at += c
    s = {"case": dict(case), "table": table,
         "begin": torch.tensor([sum(new[:r]) for r in range(len(new) + 1)], dtype=torch.int32, device=dev),
         "kv_len": torch.tensor(total, dtype=torch.int32, device=dev)}
    shape = (n_pages, page, n_kv, dim)
    for x in ("k", "v"):
        if case["op"] == "append":
            s[x] = torch.zeros(shape, dtype=torch.uint8, device=dev).view(DT[fmt]) if fmt in QMAX else torch.zeros(shape, dtype=DT[fmt], device=dev)
            # a few channels are several times the others, as keys have them
            amp = 1 + 5 * (torch.rand(n_kv, dim, generator=g, device=dev) < 0.03)
            s["new_" + x] = (torch.randn(sum(new), n_kv, dim, generator=g, device=dev) * amp).to(DT[case["src"]])
        elif fmt == "int8":
            s[x] = (torch.randn(shape, generator=g, device=dev) * 40).round_().clamp_(-127, 127).to(torch.int8)
        elif fmt == "e4m3":
            s[x] = (torch.randn(shape, generator=g, device=dev) * 140).clamp_(-448, 448).to(DT[fmt])
        else:
            s[x] = torch.randn(shape, generator=g, device=dev).to(DT[fmt])
        if fmt in QMAX:
            s[x + "_scale"] = (torch.rand(shape[:3], generator=g, device=dev) + 0.5) * (3.2 / QMAX[fmt])
        else:
            s[x + "_scale"] = None
    if case["op"] == "read":
        # the last `new` positions of each request
        s["first"] = s["kv_len"] - (s["begin"][1:] - s["begin"][:-1])
        s["tokens"] = sum(new)
    if case["op"] == "attn":
        s["q"] = torch.randn(sum(new), case["n_q"], dim, generator=g, device=dev).to(DT[case["q"]])
        s["max_new"], s["max_len"] = max(new), max(total)
        s["tree"] = _tree_masks(new, seed).to(dev) if case["tree"] else None
    return s


def _tree_masks(new, seed):
    """For each token a word whose bit j says that token j of its request is the token or one of its ancestors
    in a random tree whose root is token 0."""
    g = torch.Generator().manual_seed(int(seed))
    words = []
    for n in new:
        parent = (torch.rand(n, generator=g) * torch.arange(n)).long().tolist()
        w = [1]
        for i in range(1, n):
            w.append(w[parent[i]] | 1 << i)
        words += [x - (1 << 64) if x >> 63 else x for x in w]
    return torch.tensor(words, dtype=torch.int64)


def _prepare_sample(case, g, dev):
    n, v = case["rows"], case["vocab"]
    x = torch.randn(n, v, generator=g, device=dev) * 2.2
    hot = torch.randint(0, v, (n, 40), generator=g, device=dev)       # a few likely tokens over a broad tail
    x.scatter_add_(1, hot, torch.rand(n, 40, generator=g, device=dev) * 12)
    u = lambda: torch.rand(n, generator=g, device=dev)  # noqa: E731
    off = lambda t, value: torch.where(u() < 0.3, torch.full_like(t, value), t)  # noqa: E731 - a setting left off
    temp = 0.4 + 0.9 * u()
    if case["greedy"]:
        temp = torch.where(u() < 0.15, torch.zeros_like(temp), temp)
    return {"case": dict(case), "logits": x.to(DT[case["dtype"]]), "temperature": temp,
            "top_k": off((1 + 199 * u()).floor(), 0.0).to(torch.int32), "top_p": off(0.6 + 0.39 * u(), 1.0),
            "min_p": off(0.1 * u(), 0.0), "uniform": u()}


# ------------------------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if op == "append":
        return _own_append(state) if own else _append(state)
    if op == "read":
        return _own_read(state) if own else _read(state, state["begin"], state["first"], state["tokens"])
    if op == "attn":
        return _own_attention(state) if own else _attention(state)
    return _own_sample(state) if own else _sample(state)


def _rows(begin, count):
    """Request and index within the request of each of `count` packed tokens."""
    t = torch.arange(count, device=begin.device)
    r = torch.searchsorted(begin[1:].long(), t, right=True)
    return r, t - begin.long()[r]


def _slots(s, r, pos):
    page = s["case"]["page"]
    return s["table"].long()[r, pos // page] * page + pos % page


def _values(pool, scale, slots):
    """The values of the pool's rows at `slots`, in 32 bits."""
    flat = pool.view(torch.uint8).reshape(-1, pool.shape[2], pool.shape[3] * pool.element_size())
    x = flat[slots].view(pool.dtype).float()
    return x if scale is None else x * scale.reshape(-1, pool.shape[2])[slots][..., None]


def _read(s, begin, first, count):
    r, i = _rows(begin, count)
    slots = _slots(s, r, first.long()[r] + i)
    out = DT[s["case"]["out"]]
    return {x: _values(s[x], s[x + "_scale"], slots).to(out) for x in ("k", "v")}


def _store(s, name, slots):
    x, pool, fmt = s["new_" + name], s[name], s["case"]["fmt"]
    if fmt in QMAX:
        x = x.float()
        scale = (x.abs().amax(-1) / torch.full((), QMAX[fmt], device=x.device)).clamp_min(2.0 ** -126)
        y = x / scale[..., None]
        y = (y.round() if fmt == "int8" else y).clamp(-QMAX[fmt], QMAX[fmt]).to(DT[fmt])
        s[name + "_scale"].view(-1, pool.shape[2])[slots] = scale
    else:
        y = x.to(DT[fmt])
    pool.view(torch.uint8).view(-1, pool.shape[2], pool.shape[3] * pool.element_size())[slots] = y.view(torch.uint8)


def _append(s):
    count = s["new_k"].shape[0]
    r, i = _rows(s["begin"], count)
    first = s["kv_len"] - (s["begin"][1:] - s["begin"][:-1])
    slots = _slots(s, r, first.long()[r] + i)
    _store(s, "k", slots)
    _store(s, "v", slots)
    return _read(s, s["begin"], first, count)


def _attention(s):
    c, q = s["case"], s["q"]
    n, hk, d, group = c["n_req"], c["n_kv"], c["dim"], c["n_q"] // c["n_kv"]
    dev, m, length = q.device, s["max_new"], s["max_len"]
    begin, total = s["begin"].long(), s["kv_len"].long()
    new = begin[1:] - begin[:-1]
    pos = torch.arange(length, device=dev)
    slots = _slots(s, torch.arange(n, device=dev)[:, None], torch.minimum(pos, total[:, None] - 1))
    k, v = (_values(s[x], s[x + "_scale"], slots).transpose(1, 2) for x in ("k", "v"))       # [n, hk, keys, d]
    i = torch.arange(m, device=dev)
    at = torch.minimum(begin[:-1, None] + i, begin[1:, None] - 1)                             # [n, m]
    qs = q[at].float().view(n, m, hk, group, d).permute(0, 2, 1, 3, 4).reshape(n, hk, m * group, d)
    z = (torch.matmul(qs, k.transpose(2, 3)) * d ** -0.5).view(n, hk, m, group, length)
    p_i = ((total - new)[:, None] + i)[:, :, None]                                            # position of each query
    seen = (pos < total[:, None, None]) & (i < new[:, None])[:, :, None]
    if s["tree"] is None:
        seen = seen & (pos <= p_i)
    else:
        j = pos - (total - new)[:, None, None]
        bit = (s["tree"][at][:, :, None] >> j.clamp(0, 63)) & 1
        seen = seen & ((j < 0) | (bit == 1))
    if c["window"]:
        seen = seen & (p_i - pos < c["window"])
    seen = seen[:, None, :, None, :]
    z.masked_fill_(~seen, float("-inf"))
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    e = z.sub_(top).exp_()
    norm = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(n, hk, m * group, length), v).view(n, hk, m, group, d)
    o = torch.where(norm > 0, o / norm, torch.zeros_like(o))
    r, t = _rows(s["begin"], q.shape[0])
    out = {"out": o.permute(0, 2, 1, 3, 4)[r, t].reshape(q.shape).to(q.dtype)}
    if c["lse"]:
        out["lse"] = (norm.log() + top)[..., 0].permute(0, 2, 1, 3)[r, t].reshape(q.shape[:2])
    return out


def _sample(s):
    x = s["logits"].double()
    t, k = s["temperature"].double()[:, None], s["top_k"].long()[:, None]
    p, m, u = (s[y].double()[:, None] for y in ("top_p", "min_p", "uniform"))
    xs, order = torch.sort(x, dim=-1, descending=True, stable=True)
    greedy = t == 0
    w = ((xs - xs[:, :1]) / torch.where(greedy, torch.ones_like(t), t)).exp()
    rank = torch.arange(x.shape[1], device=x.device)
    keep = (rank < torch.where(k > 0, k, torch.full_like(k, x.shape[1]))) & (~greedy | (rank == 0))
    w = w * keep
    run_mass = w.cumsum(-1)
    keep = keep & ((rank == 0) | ((run_mass - w < p * run_mass[:, -1:]) & (w >= m)) | (p >= 1) & (w >= m))
    mass = torch.zeros_like(x).scatter_(1, order, w * keep)
    cdf = mass.cumsum(-1)
    token = (cdf <= u * cdf[:, -1:]).sum(-1)
    out = {"token": token.to(torch.int32), "prob": (mass.gather(1, token[:, None])[:, 0] / cdf[:, -1]).float()}
    if s["case"]["kept"]:
        kept = torch.zeros_like(x, dtype=torch.bool).scatter_(1, order, keep)
        out["kept"] = torch.where(kept, x.float(), torch.full((), -1e30, device=x.device))
    return out


# ------------------------------------------------------------------------------------ the package's calls

@functools.lru_cache(maxsize=None)
def _handle(n_q, n_kv, dim, page, fmt):
    """One handle (it owns the scratch) for each geometry, as a program that serves one model keeps it."""
    import block_drafter_pos_gb300 as bd
    return bd.dflash2_paged_create(bd.make_paged_config(n_q, n_kv, dim, page, fmt, max_requests=64))


def _cache(s):
    import block_drafter_pos_gb300 as bd
    return bd.paged_cache(s["k"], s["v"], s["table"], s["k_scale"], s["v_scale"])


def _own_append(s):
    import block_drafter_pos_gb300 as bd
    c, k = s["case"], s["new_k"]
    h, cache = _handle(c["n_kv"], c["n_kv"], c["dim"], c["page"], c["fmt"]), _cache(s)
    bd.dflash2_paged_write(h, cache, k, s["new_v"], s["begin"], s["kv_len"])
    out = {x: torch.empty(k.shape, dtype=DT[c["out"]], device=k.device) for x in ("k", "v")}
    bd.dflash2_paged_read(h, cache, out["k"], out["v"], s["begin"], s["kv_len"])
    return out


def _own_read(s):
    import block_drafter_pos_gb300 as bd
    c, k = s["case"], s["k"]
    h, cache = _handle(c["n_kv"], c["n_kv"], c["dim"], c["page"], c["fmt"]), _cache(s)
    out = {x: torch.empty((s["tokens"],) + k.shape[2:], dtype=DT[c["out"]], device=k.device) for x in ("k", "v")}
    bd.dflash2_paged_read(h, cache, out["k"], out["v"], s["begin"], s["kv_len"])
    return out


def _own_attention(s):
    import block_drafter_pos_gb300 as bd
    c, q = s["case"], s["q"]
    h, cache = _handle(c["n_q"], c["n_kv"], c["dim"], c["page"], c["fmt"]), _cache(s)
    out = {"out": torch.empty_like(q)}
    if c["lse"]:
        out["lse"] = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    bd.dflash2_paged_attention(h, cache, q, out["out"], s["begin"], s["kv_len"], max_new=s["max_new"], max_len=s["max_len"],
                               scale=c["dim"] ** -0.5, window=c["window"], tree_mask=s["tree"], lse=out.get("lse"))
    return out


def _own_sample(s):
    import block_drafter_pos_gb300 as bd
    x = s["logits"]
    n, dev = x.shape[0], x.device
    out = {"token": torch.empty(n, dtype=torch.int32, device=dev), "prob": torch.empty(n, dtype=torch.float32, device=dev)}
    if s["case"]["kept"]:
        out["kept"] = torch.empty(x.shape, dtype=torch.float32, device=dev)
    bd.dflash2_sample(x, s["temperature"], s["top_k"], s["top_p"], s["min_p"], s["uniform"], out["token"], prob=out["prob"],
                      kept=out.get("kept"))
    return out


# ------------------------------------------------------------------------------------ work, and the definition in 64 bits

def work(case):
    if case["op"] == "sample":
        n, v = case["rows"], case["vocab"]
        return {"bytes": n * v * (SIZE[case["dtype"]] + 4 * case["kept"]) + 28 * n, "flops": 4 * n * v}
    new, total = _lengths(case)
    hk, d, size = case["n_kv"], case["dim"], SIZE[case["fmt"]]
    row = 2 * hk * (d * size + (4 if case["fmt"] in QMAX else 0))          # one position's keys and values in the cache
    if case["op"] == "read":
        return {"bytes": sum(new) * (row + 2 * hk * d * SIZE[case["out"]]), "flops": 2 * sum(new) * hk * d}
    if case["op"] == "append":
        moved = 2 * hk * d * (SIZE[case["src"]] + SIZE[case["out"]])
        return {"bytes": sum(new) * (2 * row + moved), "flops": 8 * sum(new) * hk * d}
    w = case["window"] or 1 << 40
    keys = sum(min(t, w + n - 1) for n, t in zip(new, total))
    # query i of a chunk sees min(its position + 1, window) keys (a tree's tokens: about half of the tree less)
    full = [(min(w, t) - (t - n)) for n, t in zip(new, total)]             # queries whose window reaches back to key 0
    pairs = sum(sum(min(w, t - n + i + 1) for i in (0, n - 1)) / 2 * n if f <= 0 or f >= n else
                (t - n + 1 + w) / 2 * f + w * (n - f) for n, t, f in zip(new, total, full))
    io = sum(new) * case["n_q"] * (2 * d * SIZE[case["q"]] + 4 * case["lse"])
    return {"bytes": keys * row + io, "flops": 4 * d * case["n_q"] * pairs}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sample":
        return _exact_sample(s)
    new, total = _lengths(case)
    keys, values = ([_exact_rows(s, x, r, n, t) for r, (n, t) in enumerate(zip(new, total))] for x in ("k", "v"))
    if case["op"] != "attn":
        return {"k": torch.cat([x[t - n:] for x, n, t in zip(keys, new, total)]),
                "v": torch.cat([x[t - n:] for x, n, t in zip(values, new, total)])}
    group = case["n_q"] // case["n_kv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    at = 0
    for r, (n, t) in enumerate(zip(new, total)):
        query = torch.arange(t - n, t, device="cuda")[:, None]
        key = torch.arange(t, device="cuda")[None]
        hidden = key > query
        if s["tree"] is not None:
            word = s["tree"][at:at + n].tolist()
            hidden[:, t - n:] = torch.tensor([[not (w >> j) & 1 for j in range(n)] for w in word], device="cuda")
        if case["window"]:
            hidden = hidden | (query - key >= case["window"])
        for h in range(case["n_q"]):
            z = s["q"][at:at + n, h].double() @ keys[r][:, h // group].T / case["dim"] ** 0.5
            z[hidden] = float("-inf")
            out[at:at + n, h] = torch.softmax(z, -1) @ values[r][:, h // group]
            lse[at:at + n, h] = torch.logsumexp(z, -1)
        at += n
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


def _exact_rows(s, name, r, new, total):
    """Keys or values of request r in 64 bits, [total, heads, dim], with the new tokens in their places."""
    pages = s["table"][r].long()
    held = s[name][pages].double().flatten(0, 1)[:total]
    if s[name + "_scale"] is not None:
        held = held * s[name + "_scale"][pages].double().flatten(0, 1)[:total, :, None]
    if "new_" + name in s:
        b = int(s["begin"][r])
        x, fmt = s["new_" + name][b:b + new].double(), s["case"]["fmt"]
        if fmt == "int8":
            step = x.abs().amax(-1, keepdim=True).clamp_min(1e-300) / 127
            x = torch.round(x / step) * step
        elif fmt == "e4m3":                        # a sign, 3 bits after the leading one, exponents from -6
            step = x.abs().amax(-1, keepdim=True).clamp_min(1e-300) / 448
            y = x / step
            ulp = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
            x = torch.round(y / ulp) * ulp * step
        else:
            x = x.to(DT[fmt]).double()
        held[total - new:] = x
    return held


def _exact_sample(s):
    tokens, probs, kept = [], [], []
    for r in range(s["case"]["rows"]):
        x = s["logits"][r].double()
        t, k = float(s["temperature"][r]), int(s["top_k"][r])
        p, m, u = (float(s[y][r]) for y in ("top_p", "min_p", "uniform"))
        ids = torch.argsort(-x, stable=True)       # by logit, equal ones by id
        ids = ids[:1] if t == 0 else ids[:k] if k > 0 else ids
        w = torch.softmax(x[ids] / (t or 1.0), 0)
        if p < 1:
            before = torch.cat([w.new_zeros(1), w.cumsum(0)[:-1]])
            last = max(1, int((before < p).sum()))
            ids, w = ids[:last], w[:last]
        stay = w >= m * w[0]
        ids, w = ids[stay], w[stay]
        by_id = torch.argsort(ids)
        cdf = w[by_id].cumsum(0)
        pick = min(int((cdf <= u * cdf[-1]).sum()), len(ids) - 1)
        tokens.append(int(ids[by_id][pick]))
        probs.append(float(w[by_id][pick] / cdf[-1]))
        if s["case"]["kept"]:
            row = torch.full_like(x, -1e30)
            row[ids] = x[ids]
            kept.append(row)
    out = {"token": torch.tensor(tokens), "prob": torch.tensor(probs, dtype=torch.float64)}
    if kept:
        out["kept"] = torch.stack(kept)
    return out
