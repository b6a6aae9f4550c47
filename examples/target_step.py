"""The drafter next to a target: speculative decoding with a small random target model.

The target's layers keep their keys and values in paged int8 caches.  Prompts go through in
chunks, the first token is sampled, and every step drafts a block, runs the target over the
block (paged write and attention, one row per block position), truncates the target's rows
with the requests' sampling settings and verifies the draft against them:

    python examples/target_step.py [--steps 12] [--temperature 0.8] [--top-k 40] [--top-p 0.95]

With `--temperature 0` the tokens are those of decoding one token at a time (`--plain`), up to near-ties
of the target's logits.
"""
from __future__ import annotations

import argparse
import dataclasses
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_drafter_pos_gb300 as bd  # noqa: E402
import workloads as wk  # noqa: E402


@dataclasses.dataclass
class Settings:
    temperature: float = 0.8
    top_k: int = 40
    top_p: float = 0.95
    min_p: float = 0.0


class Target:
    """A random attention-only model of `layers` layers over the drafter's vocabulary: embedding, per layer
    norm -> q, k, v -> paged cache and attention -> output projection, final norm, LM head."""

    def __init__(self, geom, embed, lm_head, n_req, max_len, layers=2, page=16, kv_format="int8", seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hq, self.hk, self.dim, self.layers = geom.n_q_heads, geom.n_kv_heads, geom.head_dim, layers
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda") * 0.05  # noqa: E731
        width = (self.hq + 2 * self.hk) * self.dim
        self.w_qkv = [rand(geom.hidden, width) for _ in range(layers)]
        self.w_o = [rand(self.hq * self.dim, geom.hidden) for _ in range(layers)]
        self.embed, self.lm_head = embed.float(), lm_head.float()
        self.n_req, self.vocab = n_req, lm_head.shape[0]
        pages = -(-max_len // page)
        self.table = torch.randperm(n_req * pages, generator=g, device="cuda").to(torch.int32).view(n_req, pages)
        self.handle = bd.dflash2_paged_create(
            bd.make_paged_config(self.hq, self.hk, self.dim, page, kv_format, max_requests=n_req))
        self.max_len = pages * page
        self.pools = []
        for _ in range(layers):
            kv = [torch.zeros(n_req * pages, page, self.hk, self.dim, dtype=torch.int8, device="cuda") for _ in "kv"]
            scales = [torch.zeros(n_req * pages, page, self.hk, device="cuda") for _ in "kv"]
            self.pools.append(bd.paged_cache(*kv, self.table, *scales))

    @staticmethod
    def _norm(x):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)

    def forward(self, tokens, begin, kv_len, max_new):
        """Packed new tokens -> (logits fp32 [tokens, vocab], hidden states [tokens, hidden]); their keys and values
        go into the caches."""
        x = self.embed[tokens.long()]
        n = x.shape[0]
        for w_qkv, w_o, pool in zip(self.w_qkv, self.w_o, self.pools):
            qkv = (self._norm(x) @ w_qkv).to(torch.bfloat16).view(n, self.hq + 2 * self.hk, self.dim)
            q, k, v = qkv.split([self.hq, self.hk, self.hk], 1)          # rows of the fused projection, not copied
            bd.dflash2_paged_write(self.handle, pool, k, v, begin, kv_len)
            out = torch.empty(n, self.hq, self.dim, dtype=torch.bfloat16, device="cuda")
            bd.dflash2_paged_attention(self.handle, pool, q, out, begin, kv_len, max_new=max_new, max_len=self.max_len,
                                       scale=self.dim ** -0.5)
            x = x + out.view(n, -1).float() @ w_o
        h = self._norm(x)
        return h @ self.lm_head.T, h

    def close(self):
        bd.dflash2_paged_destroy(self.handle)


def _vectors(s: Settings, n):
    full = lambda v, t: torch.full((n,), v, dtype=t, device="cuda")  # noqa: E731
    return full(s.temperature, torch.float32), full(s.top_k, torch.int32), full(s.top_p, torch.float32), \
        full(s.min_p, torch.float32)


def run(steps=12, settings=Settings(), prompts=(37, 64, 90), plain=False, seed=0, force=None, watch=None):
    """Tokens of each request after its prompt (lists of at least `steps` tokens), and the mean number of
    tokens a step emitted.  plain: one token at a time; force: the tokens to feed then, in place of those sampled;
    watch: called with the logits of every plain step."""
    geom = wk.TOY
    n_req, B, P = len(prompts), geom.block, geom.block - 1
    W = wk.make_weights(geom, "bf16", seed)
    bf = lambda a: torch.from_numpy(a.view("int16")).cuda().view(torch.bfloat16)  # noqa: E731
    max_len = max(prompts) + (steps + 1) * B + 8
    target = Target(geom, bf(W["embed"]), bf(W["lm_head"]), n_req, max_len, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731

    # the prompts, in chunks of at most 48 tokens; the hidden states of the last 8 positions feed the drafter
    length = [0] * n_req
    ids = [torch.randint(0, geom.vocab - 1, (p,), generator=g, device="cuda", dtype=torch.int32) for p in prompts]
    hidden = [torch.zeros(0, geom.hidden, device="cuda") for _ in prompts]
    last = [None] * n_req
    while any(n < p for n, p in zip(length, prompts)):
        new = [min(48, p - n) for n, p in zip(length, prompts)]
        tokens = torch.cat([t[n:n + m] for t, n, m in zip(ids, length, new)])
        begin = [sum(new[:r]) for r in range(n_req + 1)]
        length = [n + m for n, m in zip(length, new)]
        logits, h = target.forward(tokens, i32(begin), i32(length), max(new))
        for r in range(n_req):
            if new[r]:
                last[r] = logits[begin[r + 1] - 1]
                hidden[r] = torch.cat([hidden[r], h[begin[r]:begin[r + 1]]])[-8:]
    # the first token of each request
    temperature, top_k, top_p, min_p = _vectors(settings, n_req)
    anchors = torch.empty(n_req, dtype=torch.int32, device="cuda")
    bd.dflash2_sample(torch.stack(last), temperature, top_k, top_p, min_p, torch.rand(n_req, generator=g, device="cuda"),
                      anchors)
    emitted = [[int(a)] for a in anchors]
    kv_len = i32(length)

    if plain:
        one = torch.arange(n_req + 1, dtype=torch.int32, device="cuda")
        for i in range(steps):
            if force is not None:
                anchors = i32([t[i] for t in force])
            kv_len += 1
            logits, _ = target.forward(anchors, one, kv_len, 1)
            if watch is not None:
                watch(logits)
            bd.dflash2_sample(logits, temperature, top_k, top_p, min_p, torch.rand(n_req, generator=g, device="cuda"), anchors)
            for e, a in zip(emitted, anchors.tolist()):
                e.append(a)
        target.close()
        return emitted, 1.0

    cap = max_len + 256
    drafter = bd.Drafter(geom, "bf16", W, n_req, cap)
    kc, vc = (torch.zeros(geom.n_layers, n_req, cap, geom.n_kv_heads, geom.head_dim, dtype=torch.int16, device="cuda")
              for _ in "kv")
    ctx_len, n_new = i32([n - 8 for n in length]), i32([8] * n_req)
    taps = torch.zeros(n_req, 8, geom.n_taps * geom.hidden, device="cuda")
    for r in range(n_req):
        taps[r] = hidden[r].repeat(1, geom.n_taps)
    z = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    cand_ids, cand_logits, gate = z(n_req, P, 16, t=torch.int32), z(n_req, P, 16), z(n_req, P, geom.rank)
    path, q_rows, status = z(n_req, P, t=torch.int32), z(n_req, P, 16), z(n_req, t=torch.int32)
    n_acc, out, n_out = z(n_req, t=torch.int32), z(n_req, B, t=torch.int32), z(n_req, t=torch.int32)
    seeds = torch.full((n_req,), 42, dtype=torch.int64, device="cuda")
    offsets = torch.arange(n_req, dtype=torch.int64, device="cuda") << 32
    block = i32([B * r for r in range(n_req + 1)])
    rows = _vectors(settings, n_req * B)
    kept, unused = z(n_req * B, geom.vocab), z(n_req * B, t=torch.int32)
    total = 0
    for _ in range(steps):
        bd.dflash2_draft_block(drafter.handle, n_req, anchors, ctx_len, n_new, taps, kc, vc, cand_ids, cand_logits, gate)
        bd.dflash2_select(drafter.handle, n_req, anchors, cand_ids, cand_logits, gate, temperature, seeds, offsets, path,
                          q_rows, None, status)
        # the target over the anchor and the proposals
        tokens = torch.cat([anchors[:, None], path], 1).view(-1)
        kv_len += B
        logits, h = target.forward(tokens, block, kv_len, B)
        # its rows, truncated as the requests ask: verify's target distribution
        bd.dflash2_sample(logits, *rows, torch.zeros(n_req * B, device="cuda"), unused, kept=kept)
        bd.dflash2_verify(drafter.handle, n_req, kept, path, cand_ids, q_rows, temperature, seeds, offsets, n_acc, out, n_out,
                          None, status)
        if status.any():
            raise RuntimeError(f"status {status.tolist()}")
        # the anchor and the accepted proposals stay in the target's cache; the rest of the block is overwritten later
        kv_len -= B - n_out
        bd.dflash2_advance(drafter.handle, n_req, out, n_out, anchors, ctx_len, n_new, offsets)
        taps.copy_(h.view(n_req, B, geom.hidden).repeat(1, 1, geom.n_taps))
        total += int(n_out.sum())
        for e, o, n in zip(emitted, out.tolist(), n_out.tolist()):
            e.extend(o[:n])
    drafter.close()
    target.close()
    return emitted, total / (steps * n_req)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=12)
    ap.add_argument("--temperature", type=float, default=0.8)
    ap.add_argument("--top-k", type=int, default=40)
    ap.add_argument("--top-p", type=float, default=0.95)
    ap.add_argument("--min-p", type=float, default=0.0)
    ap.add_argument("--plain", action="store_true", help="decode one token at a time, without the drafter")
    a = ap.parse_args()
    bd.build()
    tokens, mean = run(a.steps, Settings(a.temperature, a.top_k, a.top_p, a.min_p), plain=a.plain)
    for r, t in enumerate(tokens):
        print(f"request {r}: {t}")
    print(f"{mean:.2f} tokens a step")


if __name__ == "__main__":
    main()
