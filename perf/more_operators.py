"""Serving many samples of one prompt, as it is measured: rotary positions (of rows, and of the keys on their way into
the paged cache), the pages' bookkeeping (forking, taking, copying on write, freeing; moving a tree's accepted tokens
together), and attention of a batch whose requests share a prefix, with the prefix's keys read once for all.

`run` computes each operator in elementary torch operations (32 bits, angles in 64), or, with `own`, through the
package's entry points.
"""
import functools
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "int8": torch.int8,
      "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "int8": 1, "e4m3": 1}
QMAX = {"int8": 127.0, "e4m3": 448.0}
THETA = 1e7              # the drafter geometry's
ORIGINAL = 32768         # positions that a scaled model was trained on


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # the queries and keys of one verify block (anchor + 7 proposals): launch latency
        {"name": "rope_block", "op": "rope", "tokens": 8, "n_q": 32, "n_kv": 8, "dim": 128, "rot": 128, "layout": "half",
         "scaling": "none", "dtype": "bf16", "inverse": False, "far": 8192},
        # the queries and keys of a long prompt of a model stretched to four times its length
        {"name": "rope_prompt", "op": "rope", "tokens": 32768, "n_q": 32, "n_kv": 8, "dim": 128, "rot": 128, "layout": "half",
         "scaling": "yarn", "dtype": "bf16", "inverse": False, "far": 131072},
        # the gradient's way back through the rotation: interleaved pairs, a quarter of a head of 64, an odd number of tokens
        {"name": "rope_gradient", "op": "rope", "tokens": 9001, "n_q": 24, "n_kv": 4, "dim": 64, "rot": 16,
         "layout": "interleaved", "scaling": "linear", "dtype": "fp32", "inverse": True, "far": 30000},
        # single tokens of 64 samples into an int8 cache
        {"name": "rope_write_tokens", "op": "rope_write", "n_req": 64, "chunk": 1, "ragged": 0.5, "ctx": 4096, "n_q": 32,
         "n_kv": 8, "dim": 128, "rot": 128, "layout": "half", "scaling": "none", "page": 16, "fmt": "int8", "dtype": "bf16"},
        # five prompts' chunks of unequal lengths into an 8-bit float cache, half of each head rotated
        {"name": "rope_write_prompts", "op": "rope_write", "n_req": 5, "chunk": 6001, "ragged": 0.7, "ctx": 12000, "n_q": 32,
         "n_kv": 8, "dim": 128, "rot": 64, "layout": "half", "scaling": "yarn", "page": 64, "fmt": "e4m3", "dtype": "bf16"},
        # eight samples of one prompt: the old group freed, a new one forked, pages for its first block, one layer's tails copied
        {"name": "fork_samples", "op": "fork", "prompts": 1, "samples": 8, "prompt": 1000, "own": 8, "page": 16, "spare": 100,
         "layers": 1, "n_kv": 8, "dim": 128, "fmt": "bf16"},
        # 32 samples of each of 8 ragged prompts in a large pool of pages of one small head, two layers' tails copied
        {"name": "fork_batch", "op": "fork", "prompts": 8, "samples": 32, "prompt": 16001, "own": 700, "page": 16,
         "spare": 100000, "layers": 2, "n_kv": 1, "dim": 64, "fmt": "fp16"},
        # the accepted path of one request's tree of 33, four layers
        {"name": "keep_tree", "op": "keep", "n_req": 1, "nodes": 33, "kept": 5, "ctx": 1000, "page": 16, "layers": 4, "n_kv": 8,
         "dim": 128, "fmt": "bf16"},
        # trees of 64 of 48 requests, 16 layers
        {"name": "keep_trees", "op": "keep", "n_req": 48, "nodes": 64, "kept": 16, "ctx": 130, "page": 24, "layers": 16, "n_kv": 8,
         "dim": 128, "fmt": "fp16"},
        # a token of each of four samples of a short prompt: latency
        {"name": "shared_tokens_4", "op": "shared", "groups": 1, "n_req": 4, "chunk": 1, "prefix": 1024, "own": 60, "ragged": 0.5,
         "n_q": 32, "n_kv": 8, "dim": 128, "page": 16, "fmt": "bf16", "q": "bf16", "tree": False, "lse": False},
        # a token of each of 64 samples of one long prompt
        {"name": "shared_tokens_64", "op": "shared", "groups": 1, "n_req": 64, "chunk": 1, "prefix": 32768, "own": 1024,
         "ragged": 0.8, "n_q": 32, "n_kv": 8, "dim": 128, "page": 64, "fmt": "bf16", "q": "bf16", "tree": False, "lse": True},
        # verify blocks of 48 samples of three prompts of odd lengths, 8-bit cache: the largest
        {"name": "shared_blocks_48", "op": "shared", "groups": 3, "n_req": 48, "chunk": 8, "prefix": 30001, "own": 2000,
         "ragged": 0.6, "n_q": 32, "n_kv": 8, "dim": 128, "page": 48, "fmt": "e4m3", "q": "bf16", "tree": False, "lse": False},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["rope", "rope_write", "fork", "keep", "shared", "shared"])
    page = rng.choice([1, 8, 16, 24, 32, 48, 64, 128])
    n_kv, dim, group = rng.choice([1, 2, 4, 8]), rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 8])
    if op in ("rope", "rope_write"):
        wide = dim if op == "rope_write" else rng.choice([64, 80, 128, 192, 256])
        c = {"op": op, "n_q": n_kv * group, "n_kv": n_kv, "dim": wide, "rot": 16 * rng.randint(1, wide // 16),
             "layout": rng.choice(["half", "interleaved"]), "scaling": rng.choice(["none", "linear", "yarn"]),
             "dtype": rng.choice(["bf16", "fp16", "fp32"])}
        if op == "rope":
            c.update(tokens=min(_log_int(rng, 1, 16000), 10 ** 8 // (n_kv * (group + 1) * wide)), inverse=rng.random() < 0.5, far=_log_int(rng, 20000, 1000000))
        else:
            chunk = _log_int(rng, 1, 6000)
            c.update(n_req=_log_int(rng, 1, 5), chunk=chunk, ragged=round(rng.random() * 0.9, 2), ctx=chunk + _log_int(rng, 1, 4000),
                     page=page, fmt=rng.choice(["bf16", "fp16", "int8", "e4m3"]))
        return c
    if op == "fork":
        return {"op": op, "prompts": _log_int(rng, 1, 8), "samples": _log_int(rng, 1, 32), "prompt": _log_int(rng, 1, 8000),
                "own": _log_int(rng, 1, 700), "page": rng.choice([8, 16, 24, 32]), "spare": _log_int(rng, 10, 60000), "layers": 1,
                "n_kv": 1, "dim": dim, "fmt": rng.choice(["bf16", "fp16"])}
    if op == "keep":
        nodes = rng.randint(2, 64)
        return {"op": op, "n_req": _log_int(rng, 1, 48), "nodes": nodes, "kept": rng.randint(1, nodes), "ctx": nodes + _log_int(rng, 1, 200),
                "page": page, "layers": _log_int(rng, 1, 8), "n_kv": n_kv, "dim": dim, "fmt": rng.choice(["bf16", "fp16"])}
    kind = rng.choice(["token", "block", "tree", "chunk"])
    groups = _log_int(rng, 1, 6)
    n_req = groups * _log_int(rng, 1, 16)
    chunk = {"token": 1, "block": rng.randint(2, 16), "tree": rng.randint(2, 64), "chunk": rng.randint(65, 300)}[kind]
    n_kv = max(1, n_kv // 2) if kind in ("tree", "chunk") else n_kv
    prefix = _log_int(rng, 1, 30000)
    # no drawn case costs more than the largest listed one: heads * queries * keys
    own_len = chunk + _log_int(rng, 1, 1000)
    prefix = max(1, min(prefix, 48 * 8 * 32 * 27000 // (n_req * chunk * n_kv * group) - own_len))
    fmt = rng.choice(["bf16", "fp16", "int8", "e4m3"])
    return {"op": op, "groups": groups, "n_req": n_req, "chunk": chunk, "prefix": prefix, "own": own_len,
            "ragged": round(rng.random() * 0.9, 2), "n_q": n_kv * group, "n_kv": n_kv, "dim": dim, "page": page, "fmt": fmt,
            "q": fmt if fmt in ("bf16", "fp16") else rng.choice(["bf16", "fp16"]), "tree": kind == "tree", "lse": rng.random() < 0.5}


def _cut(case, n, count):
    """Lengths of `count` requests: the first one's is n, the others' fall by up to the share `ragged`."""
    return [max(1, int(n * (1 - case["ragged"] * ((r * 5) % count) / count))) for r in range(count)]


def _tokens(case):
    """New tokens and cache lengths of each request."""
    if case["op"] == "keep":
        return [case["nodes"]] * case["n_req"], [case["ctx"] + (r * 7) % 11 for r in range(case["n_req"])]
    if case["op"] == "rope_write":
        new = _cut(case, case["chunk"], case["n_req"])
        return new, [max(n, t) for n, t in zip(new, _cut(case, case["ctx"], case["n_req"]))]
    new, per = [case["chunk"]] * case["n_req"], case["n_req"] // case["groups"]
    own_len = [max(case["chunk"], t) for t in _cut(case, case["own"], case["n_req"])]
    return new, [_prefixes(case)[r // per] + t for r, t in enumerate(own_len)]


def _prefixes(case):
    return [max(1, case["prefix"] - g * (case["prefix"] // 9)) for g in range(case["groups"])]


def _prompts(case):
    return [max(1, case["prompt"] - p * (case["prompt"] // 11)) for p in range(case["prompts"])]


# ------------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    s = {"case": dict(case)}
    rand = lambda *shape: torch.randn(*shape, generator=g, device=dev)  # noqa: E731
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    if case["op"] == "rope":
        t = DT[case["dtype"]]
        s["positions"] = torch.randint(0, case["far"], (case["tokens"],), generator=g, device=dev).to(torch.int32)
        s["q"], s["k"] = (rand(case["tokens"], h, case["dim"]).to(t) for h in (case["n_q"], case["n_kv"]))
        return s
    if case["op"] == "fork":
        return _prepare_fork(case, s, rand, i32, torch.randperm(1 << 20, generator=g, device=dev))
    new, total = _tokens(case)
    page, n_kv, dim, fmt = case["page"], case["n_kv"], case["dim"], case["fmt"]
    counts = [-(-t // page) for t in total]
    # a request's leading pages that it shares with the first of its group (whole pages of the prefix)
    per = case["n_req"] // case["groups"] if case["op"] == "shared" else 1
    shared = [_prefixes(case)[r // per] // page if r % per else 0 for r in range(len(new))] if case["op"] == "shared" else [0] * len(new)
    n_pages = sum(counts) - sum(shared) + 3
    ids = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)      # pages in no order, as a pool's
    table = torch.zeros(case["n_req"], max(counts), dtype=torch.int32, device=dev)
    at = 0
    for r, (c, h) in enumerate(zip(counts, shared)):
        table[r, :h] = table[r - r % per, :h]
        table[r, h:c] = ids[at:at + c - h]
        at += c - h
    s["table"], s["kv_len"] = table, i32(total)
    s["begin"] = i32([sum(new[:r]) for r in range(len(new) + 1)])
    layers = (case["layers"],) if case["op"] == "keep" else ()
    shape = layers + (n_pages, page, n_kv, dim)
    for x in ("k", "v"):
        s[x + "_scale"] = (torch.rand(shape[:-1], generator=g, device=dev) + 0.5) * (3.2 / QMAX[fmt]) if fmt in QMAX else None
        if fmt == "int8":
            s[x] = (rand(*shape) * 40).round_().clamp_(-127, 127).to(torch.int8)
        elif fmt == "e4m3":
            s[x] = (rand(*shape) * 140).clamp_(-448, 448).to(DT[fmt])
        else:
            s[x] = torch.empty(shape, dtype=DT[fmt], device=dev).normal_(generator=g)
    if case["op"] == "rope_write":
        for x, h in (("q", case["n_q"]), ("new_k", n_kv), ("new_v", n_kv)):
            s[x] = rand(sum(new), h, dim).to(DT[case["dtype"]])
    elif case["op"] == "keep":
        # the root and a path of accepted nodes: ascending, never the same twice
        order = torch.rand(case["n_req"], case["nodes"], generator=g, device=dev)
        order[:, 0] = -1
        s["keep"] = order.argsort(1)[:, :case["kept"]].sort(1).values.to(torch.int32)
        s["n_keep"] = torch.randint(1, case["kept"] + 1, (case["n_req"],), generator=g, device=dev).to(torch.int32)
    else:
        s["q"] = rand(sum(new), case["n_q"], dim).to(DT[case["q"]])
        s["group_begin"], s["prefix_len"] = i32([per * x for x in range(case["groups"] + 1)]), i32(_prefixes(case))
        # the page in which a prefix ends is each request's own, with the same rows
        for r, h in enumerate(shared):
            if r % per and h < counts[r]:
                for x in (y for y in ("k", "v", "k_scale", "v_scale") if s[y] is not None):
                    raw = s[x].view(torch.uint8)
                    raw[int(table[r, h])] = raw[int(table[r - r % per, h])]
        s["tree"] = _tree_masks(new, seed).to(dev) if case["tree"] else None
        s["max_new"], s["max_len"], s["max_prefix"] = max(new), max(total), max(_prefixes(case))
        s["max_group"], s["max_own"] = per * case["chunk"], max(t - _prefixes(case)[r // per] for r, t in enumerate(total))
    return s


def _prepare_fork(case, s, rand, i32, order):
    prompts, page = _prompts(case), case["page"]
    n, samples = case["prompts"], case["samples"]
    rows = n * (1 + samples)
    held = [-(-t // page) for t in prompts]
    width = max(-(-(t + case["own"]) // page) for t in prompts)
    n_pages = sum(held) + samples * sum(-(-(t + case["own"]) // page) - t // page for t in prompts) + case["spare"]
    dev = order.device
    ids = order[order < n_pages] if n_pages <= order.numel() else torch.arange(n_pages, device=dev).flip(0)
    s["table"] = torch.full((rows, width), -1, dtype=torch.int32, device=dev)
    s["ref"] = torch.zeros(n_pages, dtype=torch.int32, device=dev)
    at = 0
    for r, h in enumerate(held):
        s["table"][r, :h] = ids[at:at + h]
        at += h
    s["ref"][ids[:at]] = 1
    s["kv_len"] = i32(prompts + [0] * (n * samples))
    parents = [p for p in range(n) for _ in range(samples)]
    s["parent"], s["child"] = i32(parents), i32(list(range(n, rows)))
    s["freed"] = i32(prompts + [0] * (n * samples))                                # the samples' lengths once they are done,
    s["grown"] = i32(prompts + [prompts[p] + case["own"] for p in parents])        # and with their first block
    s["copies"] = torch.zeros(3, rows, dtype=torch.int32, device=dev)
    shape = (case["layers"], n_pages, page, case["n_kv"], case["dim"])
    for x in ("k", "v"):
        s[x] = torch.empty(shape, dtype=DT[case["fmt"]], device=dev)
        for layer in range(case["layers"]):
            # the prompts' pages; the others hold nothing yet
            s[x][layer].zero_()
            s[x][layer][ids[:at]] = rand(at, *shape[2:]).to(DT[case["fmt"]])
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


# ------------------------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if op == "rope":
        return _own_rope(state) if own else _rope(state)
    if op == "rope_write":
        return _own_rope_write(state) if own else _rope_write(state)
    if op == "fork":
        return _own_fork(state) if own else _fork(state)
    if op == "keep":
        return _own_keep(state) if own else _keep(state)
    return _own_shared(state) if own else _shared(state)


def _frequencies(c, device):
    """Radians per position of each pair (64 bits), and the factor of the rotated channels."""
    i = torch.arange(c["rot"] // 2, dtype=torch.float64, device=device)
    f = THETA ** (-2 * i / c["rot"])
    if c["scaling"] == "linear":
        return f / 4, 1.0
    if c["scaling"] == "yarn":       # pairs that turn often keep their frequency, those that turn less than once are stretched
        at = lambda turns: c["rot"] * math.log(ORIGINAL / (turns * 2 * math.pi)) / (2 * math.log(THETA))  # noqa: E731
        lo, hi = max(math.floor(at(32)), 0), min(math.ceil(at(1)), c["rot"] - 1)
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return f / 4 * ramp + f * (1 - ramp), 0.1 * math.log(4) + 1
    return f, 1.0


def _turn(c, x, positions, inverse):
    """Rows x [tokens, heads, dim], rotated, in 32 bits."""
    f, amplitude = _frequencies(c, x.device)
    angle = positions.double()[:, None] * f
    cos, sin = (angle.cos() * amplitude).float()[:, None], (angle.sin() * (-amplitude if inverse else amplitude)).float()[:, None]
    x = x.float()
    r, half = c["rot"], c["rot"] // 2
    if c["layout"] == "half":
        a, b = x[..., :half], x[..., half:r]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., r:]], -1)
    a, b = x[..., :r:2], x[..., 1:r:2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., r:]], -1)


def _rope(s):
    c = s["case"]
    return {x: _turn(c, s[x], s["positions"], c["inverse"]).to(s[x].dtype) for x in ("q", "k")}


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


def _rope_write(s):
    c, q = s["case"], s["q"]
    r, i = _rows(s["begin"], q.shape[0])
    pos = (s["kv_len"] - (s["begin"][1:] - s["begin"][:-1])).long()[r] + i
    slots = _slots(s, r, pos)
    out = {"q": _turn(c, q, pos, False).to(q.dtype)}
    for name, x in (("k", _turn(c, s["new_k"], pos, False)), ("v", s["new_v"].float())):
        pool, fmt = s[name], c["fmt"]
        if fmt in QMAX:
            scale = (x.abs().amax(-1) / torch.full((), QMAX[fmt], device=x.device)).clamp_min(2.0 ** -126)
            y = x / scale[..., None]
            y = (y.round() if fmt == "int8" else y).clamp(-QMAX[fmt], QMAX[fmt]).to(DT[fmt])
            s[name + "_scale"].view(-1, pool.shape[2])[slots] = scale
        else:
            y = x.to(DT[fmt])
        pool.view(torch.uint8).view(-1, pool.shape[2], pool.shape[3] * pool.element_size())[slots] = y.view(torch.uint8)
        out[name] = _values(pool, s[name + "_scale"], slots).to(q.dtype)
    return out


def _resize(s, new):
    """Pages for lengths `new`: taken (the lowest free ones, by row and column) or given back; a shared page that a
    row would write to is replaced, and noted for copying, but for the first row where every holder grows."""
    table, ref, old, page = s["table"], s["ref"], s["kv_len"], s["case"]["page"]
    n = ref.numel()
    have, need = (old + page - 1) // page, (new + page - 1) // page
    grow = new > old
    tail = table.gather(1, (have - 1).clamp_min(0).long()[:, None])[:, 0].long()
    tailed = grow & (old % page > 0)
    holders = ref[tail.clamp_min(0)]
    same = (tail[:, None] == tail) & tailed[:, None] & tailed
    first = ~same.tril(-1).any(1)
    renew = tailed & (holders > 1) & ~(first & (same.sum(1) >= holders))
    want = torch.where(grow, need - have, torch.zeros_like(have)) + renew
    free = ref == 0
    served = (want == 0) | (want.cumsum(0) <= free.sum())
    col = torch.arange(table.shape[1], device=table.device)
    fresh = (grow[:, None] & (col >= have[:, None]) & (col < need[:, None]) | renew[:, None] & (col == have[:, None] - 1)) & served[:, None]
    gone = (col >= need[:, None]) & (col < have[:, None])
    rank = free.cumsum(0)
    ids = torch.full((n + 1,), -1, dtype=torch.int32, device=table.device)
    ids.scatter_(0, torch.where(free, rank - 1, torch.full_like(rank, n)), torch.arange(n, dtype=torch.int32, device=table.device))
    taken = ids[(fresh.flatten().cumsum(0) - 1).clamp_min(0)].view(table.shape)
    renewed = renew & served
    ref.scatter_add_(0, table.clamp_min(0).long().flatten(), -(gone.flatten().to(torch.int32)))
    ref.scatter_add_(0, tail.clamp_min(0), -renewed.to(torch.int32))
    ref += (free & (rank <= fresh.sum())).to(torch.int32)
    none = torch.full_like(old, -1)
    dst = taken.gather(1, (have - 1).clamp_min(0).long()[:, None])[:, 0]
    s["copies"].copy_(torch.stack([torch.where(renewed, tail.to(torch.int32), none), torch.where(renewed, dst, none),
                                   torch.where(renewed, old % page, torch.zeros_like(old))]))
    table.copy_(torch.where(fresh, taken, torch.where(gone, torch.full_like(table, -1), table)))
    old.copy_(torch.where(served, new, old))


def _fork(s):
    table, ref, kv_len, page = s["table"], s["ref"], s["kv_len"], s["case"]["page"]
    _resize(s, s["freed"])
    parent, child = s["parent"].long(), s["child"].long()
    held = torch.arange(table.shape[1], device=table.device) < ((kv_len[parent] + page - 1) // page)[:, None]
    pages = table[parent]
    ref.scatter_add_(0, pages.clamp_min(0).long().flatten(), held.flatten().to(torch.int32))
    table[child] = torch.where(held, pages, table[child])
    kv_len[child] = kv_len[parent]
    _resize(s, s["grown"])
    # a sample without a tail to copy copies its last page onto itself
    src, dst, rows = (x.long() for x in s["copies"][:, child])
    last = table[child].gather(1, ((kv_len[child] - 1) // page).long()[:, None])[:, 0].long()
    src, dst = torch.where(src < 0, last, src), torch.where(dst < 0, last, dst)
    keep = (torch.arange(page, device=table.device) < rows[:, None])[:, :, None, None]
    for x in ("k", "v"):
        s[x][:, dst] = torch.where(keep, s[x][:, src], s[x][:, dst])
    return {x: s[x] for x in ("table", "ref", "kv_len", "copies", "k", "v")}


def _keep(s):
    page = s["case"]["page"]
    start = (s["kv_len"] - (s["begin"][1:] - s["begin"][:-1])).long()[:, None]
    r = torch.arange(start.shape[0], device=start.device)[:, None]
    j = torch.arange(s["keep"].shape[1], device=start.device)
    # (places past the accepted tokens take themselves)
    src = _slots(s, r, start + torch.where(j < s["n_keep"][:, None], s["keep"].long(), j))
    dst = _slots(s, r, start + j)
    for x in ("k", "v"):
        flat = s[x].view(s[x].shape[0], -1, *s[x].shape[3:])
        flat[:, dst] = flat[:, src]
    return {"k": s["k"], "v": s["v"], "kv_len": (start[:, 0] + s["n_keep"]).to(torch.int32)}


def _shared(s):
    c, q = s["case"], s["q"]
    n, hk, d, group, m = c["n_req"], c["n_kv"], c["dim"], c["n_q"] // c["n_kv"], c["chunk"]
    dev, per = q.device, c["n_req"] // c["groups"]
    total, prefix = s["kv_len"].long(), s["prefix_len"].long().repeat_interleave(per)
    first = torch.arange(0, n, per, device=dev)[:, None]
    # the prefixes, once for each group: [groups, hk, per * m * group, keys]
    pos = torch.arange(s["max_prefix"], device=dev)
    slots = _slots(s, first, torch.minimum(pos, s["prefix_len"].long()[:, None] - 1))
    k, v = (_values(s[x], s[x + "_scale"], slots).transpose(1, 2) for x in ("k", "v"))
    qs = q.float().view(n, m, hk, group, d)
    qg = qs.view(c["groups"], per * m, hk, group, d).permute(0, 2, 1, 3, 4).reshape(c["groups"], hk, per * m * group, d)
    z = torch.matmul(qg, k.transpose(2, 3)).mul_(d ** -0.5)
    z.masked_fill_((pos >= s["prefix_len"].long()[:, None])[:, None, None], float("-inf"))
    top_p = z.amax(-1, keepdim=True)
    e = z.sub_(top_p).exp_()
    sum_p, o_p = e.sum(-1, keepdim=True), torch.matmul(e, v)
    back = lambda x: x.view(c["groups"], hk, per, m, group, -1).permute(0, 2, 1, 3, 4, 5).reshape(n, hk, m, group, -1)  # noqa: E731
    top_p, sum_p, o_p = back(top_p), back(sum_p), back(o_p)
    # each request's own keys
    own_len = total - prefix
    pos = torch.arange(s["max_own"], device=dev)
    slots = _slots(s, torch.arange(n, device=dev)[:, None], prefix[:, None] + torch.minimum(pos, own_len[:, None] - 1))
    k, v = (_values(s[x], s[x + "_scale"], slots).transpose(1, 2) for x in ("k", "v"))
    qr = qs.permute(0, 2, 1, 3, 4).reshape(n, hk, m * group, d)
    z = torch.matmul(qr, k.transpose(2, 3)).mul_(d ** -0.5).view(n, hk, m, group, -1)
    i = torch.arange(m, device=dev)[:, None]
    j = pos - (own_len - m)[:, None, None]                                     # key j of the new tokens
    if s["tree"] is None:
        seen = j <= i
    else:
        seen = (j < 0) | ((s["tree"].view(n, m)[:, :, None] >> j.clamp(0, 63)) & 1 == 1)
    seen = seen & (pos < own_len[:, None, None])
    z.masked_fill_(~seen[:, None, :, None], float("-inf"))
    top = torch.maximum(z.amax(-1, keepdim=True), top_p)
    e = z.sub_(top).exp_()
    f = (top_p - top).exp()
    norm = e.sum(-1, keepdim=True) + sum_p * f
    o = (torch.matmul(e.view(n, hk, m * group, -1), v).view(n, hk, m, group, d) + o_p * f) / norm
    out = {"out": o.permute(0, 2, 1, 3, 4).reshape(q.shape).to(q.dtype)}
    if c["lse"]:
        out["lse"] = (norm.log() + top)[..., 0].permute(0, 2, 1, 3).reshape(q.shape[:2])
    return out


# ------------------------------------------------------------------------------------ the package's calls

@functools.lru_cache(maxsize=None)
def _plan(rot, layout, scaling):
    import block_drafter_pos_gb300 as bd
    return bd.make_rope(rot, THETA, interleaved=layout == "interleaved", scaling=scaling, factor=4.0, original_len=ORIGINAL)


@functools.lru_cache(maxsize=None)
def _handle(n_q, n_kv, dim, page, fmt):
    """One handle (it owns the scratch) for each geometry, as a program that serves one model keeps it."""
    import block_drafter_pos_gb300 as bd
    return bd.dflash2_paged_create(bd.make_paged_config(n_q, n_kv, dim, page, fmt, max_requests=128))


def _own_rope(s):
    import block_drafter_pos_gb300 as bd
    c = s["case"]
    out = {x: torch.empty_like(s[x]) for x in ("q", "k")}
    bd.dflash2_rope(_plan(c["rot"], c["layout"], c["scaling"]), s["q"], out["q"], s["positions"], k=s["k"], k_out=out["k"],
                    inverse=c["inverse"])
    return out


def _own_rope_write(s):
    import block_drafter_pos_gb300 as bd
    c, q = s["case"], s["q"]
    h = _handle(c["n_q"], c["n_kv"], c["dim"], c["page"], c["fmt"])
    cache = bd.paged_cache(s["k"], s["v"], s["table"], s["k_scale"], s["v_scale"])
    out = {"q": torch.empty_like(q), "k": torch.empty_like(s["new_k"]), "v": torch.empty_like(s["new_v"])}
    bd.dflash2_paged_rope_write(h, _plan(c["rot"], c["layout"], c["scaling"]), cache, q, out["q"], s["new_k"], s["new_v"],
                                s["begin"], s["kv_len"])
    bd.dflash2_paged_read(h, cache, out["k"], out["v"], s["begin"], s["kv_len"])
    return out


def _caches(s):
    import block_drafter_pos_gb300 as bd
    return [bd.paged_cache(s["k"][layer], s["v"][layer], s["table"]) for layer in range(s["case"]["layers"])]


def _own_fork(s):
    import block_drafter_pos_gb300 as bd
    c = s["case"]
    h = _handle(c["n_kv"], c["n_kv"], c["dim"], c["page"], c["fmt"])
    pool = bd.page_pool(s["table"], s["ref"], c["page"])
    bd.dflash2_pages_resize(pool, s["kv_len"], s["freed"], s["copies"])
    bd.dflash2_pages_fork(pool, s["parent"], s["child"], s["kv_len"])
    bd.dflash2_pages_resize(pool, s["kv_len"], s["grown"], s["copies"])
    bd.dflash2_pages_copy(h, _caches(s), s["copies"])
    return {x: s[x] for x in ("table", "ref", "kv_len", "copies", "k", "v")}


def _own_keep(s):
    import block_drafter_pos_gb300 as bd
    c = s["case"]
    h = _handle(c["n_kv"], c["n_kv"], c["dim"], c["page"], c["fmt"])
    out = torch.empty_like(s["kv_len"])
    bd.dflash2_paged_keep(h, _caches(s), s["begin"], s["kv_len"], s["keep"], s["n_keep"], kv_out=out)
    return {"k": s["k"], "v": s["v"], "kv_len": out}


def _own_shared(s):
    import block_drafter_pos_gb300 as bd
    c, q = s["case"], s["q"]
    h = _handle(c["n_q"], c["n_kv"], c["dim"], c["page"], c["fmt"])
    cache = bd.paged_cache(s["k"], s["v"], s["table"], s["k_scale"], s["v_scale"])
    out = {"out": torch.empty_like(q)}
    if c["lse"]:
        out["lse"] = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    work = torch.empty(bd.dflash2_paged_shared_bytes(h, q.shape[0]), dtype=torch.uint8, device=q.device)
    bd.dflash2_paged_attention_shared(h, cache, q, out["out"], s["begin"], s["kv_len"], s["group_begin"], s["prefix_len"], work,
                                      max_new=s["max_new"], max_len=s["max_len"], max_group=s["max_group"],
                                      max_prefix=s["max_prefix"], scale=c["dim"] ** -0.5, tree_mask=s["tree"], lse=out.get("lse"))
    return out


# ------------------------------------------------------------------------------------ work, and the definition in 64 bits

def work(case):
    size = SIZE[case.get("dtype") or case["fmt"]]
    if case["op"] == "rope":
        elements = case["tokens"] * (case["n_q"] + case["n_kv"]) * case["dim"]
        return {"bytes": 2 * elements * size + 4 * case["tokens"], "flops": 3 * elements * case["rot"] / case["dim"]}
    if case["op"] == "fork":
        prompts, page, samples = _prompts(case), case["page"], case["samples"]
        tails = samples * sum(t % page for t in prompts)
        pages = sum(-(-t // page) + samples * -(-(t + case["own"]) // page) for t in prompts)
        n_pages = sum(-(-t // page) for t in prompts) + samples * sum(-(-(t + case["own"]) // page) - t // page for t in prompts) + case["spare"]
        return {"bytes": case["layers"] * tails * 4 * case["n_kv"] * case["dim"] * size + 8 * pages + 4 * n_pages, "flops": 0}
    new, total = _tokens(case)
    hk, d = case["n_kv"], case["dim"]
    row = 2 * hk * (d * SIZE[case["fmt"]] + (4 if case["fmt"] in QMAX else 0))       # one position's keys and values in the cache
    if case["op"] == "keep":
        # half of the longest path on average; a fraction of it is in place already
        return {"bytes": case["layers"] * case["n_req"] * (1 + case["kept"]) * row, "flops": 0}
    if case["op"] == "rope_write":
        return {"bytes": sum(new) * (2 * row + (2 * case["n_q"] + 4 * hk) * d * size), "flops": 3 * sum(new) * (case["n_q"] + hk) * case["rot"]}
    per = case["n_req"] // case["groups"]
    keys = sum(_prefixes(case)) + sum(t - _prefixes(case)[r // per] for r, t in enumerate(total))
    pairs = sum(n * (t - (n - 1) / 2) for n, t in zip(new, total))
    io = sum(new) * case["n_q"] * (2 * d * SIZE[case["q"]] + 4 * case["lse"])
    return {"bytes": keys * row + io, "flops": 4 * d * case["n_q"] * pairs}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return {x: _exact_turn(case, s[x], s["positions"], -1 if case["inverse"] else 1) for x in ("q", "k")}
    if case["op"] == "fork":
        return _exact_fork(s)
    if case["op"] == "keep":
        return _exact_keep(s)
    new, total = _tokens(case)
    if case["op"] == "rope_write":
        pos = torch.cat([torch.arange(t - n, t, device="cuda") for n, t in zip(new, total)])
        return {"q": _exact_turn(case, s["q"], pos, 1), "k": _exact_held(case, _exact_turn(case, s["new_k"], pos, 1)),
                "v": _exact_held(case, s["new_v"].double())}
    keys, values = ([_exact_rows(s, x, r, t) for r, t in enumerate(total)] for x in ("k", "v"))
    group, at = case["n_q"] // case["n_kv"], 0
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    for r, (n, t) in enumerate(zip(new, total)):
        hidden = torch.arange(t, device="cuda")[None] > torch.arange(t - n, t, device="cuda")[:, None]
        if s["tree"] is not None:
            word = s["tree"][at:at + n].tolist()
            hidden[:, t - n:] = torch.tensor([[not (w >> j) & 1 for j in range(n)] for w in word], device="cuda")
        for h in range(case["n_q"]):
            z = s["q"][at:at + n, h].double() @ keys[r][:, h // group].T / case["dim"] ** 0.5
            z[hidden] = float("-inf")
            out[at:at + n, h] = torch.softmax(z, -1) @ values[r][:, h // group]
            lse[at:at + n, h] = torch.logsumexp(z, -1)
        at += n
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


def _exact_turn(c, x, positions, sign):
    """The rotated channels as complex numbers times a unit number."""
    n, half = c["rot"], c["rot"] // 2
    rate = torch.tensor([_exact_rate(c, i) for i in range(half)], dtype=torch.float64, device=x.device)
    gain = 1 + 0.1 * math.log(4) if c["scaling"] == "yarn" else 1.0
    angle = sign * positions.double()[:, None] * rate
    unit = torch.polar(torch.full_like(angle, gain), angle)[:, None]
    y = x.double().clone()
    re, im = (slice(0, half), slice(half, n)) if c["layout"] == "half" else (slice(0, n, 2), slice(1, n, 2))
    z = torch.complex(y[..., re], y[..., im]) * unit
    y[..., re], y[..., im] = z.real, z.imag
    return y


def _exact_rate(c, i):
    f = math.exp(-2 * i / c["rot"] * math.log(THETA))
    if c["scaling"] == "none":
        return f
    if c["scaling"] == "linear":
        return f / 4
    pair = lambda turns: math.log(ORIGINAL / (2 * math.pi * turns)) / math.log(THETA) * c["rot"] / 2  # noqa: E731
    lo, hi = max(0, math.floor(pair(32))), min(c["rot"] - 1, math.ceil(pair(1)))
    share = min(1.0, max(0.0, (i - lo) / (hi - lo if hi > lo else 1e-3)))
    return f * (1 - share) + f / 4 * share


def _exact_held(c, x):
    """Values x as the cache holds them."""
    if c["fmt"] == "int8":
        step = x.abs().amax(-1, keepdim=True).clamp_min(1e-300) / 127
        return torch.round(x / step) * step
    if c["fmt"] == "e4m3":                         # a sign, 3 bits after the leading one, exponents from -6
        step = x.abs().amax(-1, keepdim=True).clamp_min(1e-300) / 448
        y = x / step
        ulp = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
        return torch.round(y / ulp) * ulp * step
    return x.to(DT[c["fmt"]]).double()


def _exact_rows(s, name, r, total):
    """Keys or values of request r in 64 bits, [total, heads, dim]."""
    pages = s["table"][r, :-(-total // s["case"]["page"])].long()
    held = s[name].view(torch.uint8)[pages].view(s[name].dtype).double().flatten(0, 1)[:total]
    if s[name + "_scale"] is not None:
        held = held * s[name + "_scale"][pages].double().flatten(0, 1)[:total, :, None]
    return held


def _exact_fork(s):
    """Row by row on the host: the integers have no value in 64 bits, the copied pools do."""
    c = s["case"]
    page, table, ref = c["page"], s["table"].tolist(), s["ref"].tolist()
    free = [p for p, h in enumerate(ref) if h == 0]
    at = 0
    k, v = s["k"].double(), s["v"].double()
    for parent, child in zip(s["parent"].tolist(), s["child"].tolist()):
        length = int(s["kv_len"][parent])
        end = length + c["own"]
        fresh = -(-end // page) - length // page
        pages, at = free[at:at + fresh], at + fresh
        if length % page:
            for pool in (k, v):
                pool[:, pages[0], :length % page] = pool[:, table[parent][length // page], :length % page]
    return {"table": None, "ref": None, "kv_len": None, "copies": None, "k": k, "v": v}


def _exact_keep(s):
    page = s["case"]["page"]
    k, v = s["k"].double(), s["v"].double()
    n = s["begin"][1:] - s["begin"][:-1]
    for r in range(s["case"]["n_req"]):
        start, row = int(s["kv_len"][r] - n[r]), s["table"][r].tolist()
        for j in range(int(s["n_keep"][r])):
            a, b = start + int(s["keep"][r, j]), start + j
            for pool in (k, v):
                pool[:, row[b // page], b % page] = pool[:, row[a // page], a % page].clone()
    return {"k": k, "v": v, "kv_len": None}
