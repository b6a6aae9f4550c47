"""Several samples of one prompt: a small random target model with rotary positions whose samples share the prompt's pages.

The prompt goes through once.  Its samples are forked from it (no page is copied), and every step takes the pages that the new
tokens need, copies the prompt's last, partly filled page for the samples that write to it, turns queries and keys by their
positions on the way into the paged cache, attends over the shared prompt and each sample's own tokens, and samples the next
tokens.  At the end all pages are given back:

    python examples/shared_prompt.py [--samples 4] [--steps 12] [--temperature 0.9]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_drafter_pos_gb300 as bd  # noqa: E402


class Target:
    """A random attention-only model: embedding, per layer norm -> q, k, v -> turned and written, attention -> output
    projection; final norm, LM head.  Its layers' pools go by one page table."""

    def __init__(self, rows, n_pages, width, layers=2, vocab=4096, hidden=256, hq=8, hk=2, dim=64, page=16, kv_format="bf16", seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda") * 0.08  # noqa: E731
        self.hq, self.hk, self.dim, self.page, self.vocab = hq, hk, dim, page, vocab
        self.w_qkv = [rand(hidden, (hq + 2 * hk) * dim) for _ in range(layers)]
        self.w_o = [rand(hq * dim, hidden) for _ in range(layers)]
        self.embed, self.head = torch.randn(vocab, hidden, generator=g, device="cuda"), rand(hidden, vocab)
        self.rope = bd.make_rope(dim, theta=1e4, scaling="yarn", factor=4.0, original_len=256)
        self.handle = bd.dflash2_paged_create(bd.make_paged_config(hq, hk, dim, page, kv_format, max_requests=rows))
        i32 = lambda *s, v=0: torch.full(s, v, dtype=torch.int32, device="cuda")  # noqa: E731
        self.table, self.ref, self.kv_len = i32(rows, width, v=-1), i32(n_pages), i32(rows)
        self.copies, self.status = i32(3, rows), i32(rows)
        self.pages = bd.page_pool(self.table, self.ref, page, self.handle)
        kv = lambda: torch.zeros(n_pages, page, hk, dim, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.pools = [(kv(), kv()) for _ in range(layers)]
        self.caches = self.caches_of(0, rows)
        self.max_len = width * page

    def caches_of(self, first, last):
        """The layers' caches for rows first .. last - 1 of the page table."""
        return [bd.paged_cache(k, v, self.table[first:last]) for k, v in self.pools]

    def resize(self, new_len):
        """Brings all rows to new_len positions; raises if the pool is too small."""
        bd.dflash2_pages_resize(self.pages, self.kv_len, new_len, self.copies, self.status)
        bd.dflash2_pages_copy(self.handle, self.caches, self.copies)
        if self.status.any():
            raise RuntimeError(f"status {self.status.tolist()}")

    def forward(self, caches, tokens, begin, kv_len, max_new, attend, positions=None):
        """Packed new tokens of the caches' rows -> logits; attend(cache, q, out) is the attention's call."""
        norm = lambda x: x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)  # noqa: E731
        x, n = self.embed[tokens.long()], tokens.numel()
        for w_qkv, w_o, cache in zip(self.w_qkv, self.w_o, caches):
            qkv = (norm(x) @ w_qkv).to(torch.bfloat16).view(n, self.hq + 2 * self.hk, self.dim)
            q, k, v = qkv.split([self.hq, self.hk, self.hk], 1)            # rows of the fused projection, not copied
            bd.dflash2_paged_rope_write(self.handle, self.rope, cache, q, q, k, v, begin, kv_len, positions=positions)
            out = torch.empty(n, self.hq, self.dim, dtype=torch.bfloat16, device="cuda")
            attend(cache, q, out)
            x = x + out.view(n, -1).float() @ w_o
        return norm(x) @ self.head

    def close(self):
        bd.dflash2_paged_destroy(self.handle)


def run(samples=4, steps=12, prompt=45, temperature=0.9, top_k=50, shared="auto", seed=0, force=None, watch=None):
    """Tokens of each sample after the prompt, and how many pages were held at most.  shared: "auto", "together", "apart", or None
    for a call that knows nothing of the prefix.  force: the tokens to feed in place of those sampled; watch: called with the
    logits of every step."""
    page, rows = 16, samples + 1
    width = -(-(prompt + steps + 1) // page)
    t = Target(rows, rows * width, width, seed=seed, page=page)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    scale = t.dim ** -0.5
    # the prompt, in row 0
    ids = torch.randint(0, t.vocab, (prompt,), generator=g, device="cuda", dtype=torch.int32)
    t.resize(i32([prompt] + [0] * samples))
    begin, length = i32([0, prompt]), i32([prompt])
    one = lambda cache, q, out: bd.dflash2_paged_attention(t.handle, cache, q, out, begin, length, max_new=prompt,  # noqa: E731
                                                           max_len=t.max_len, scale=scale)
    logits = t.forward(t.caches_of(0, 1), ids, begin, length, prompt, one)[-1:]
    # its samples: rows 1 .., holders of the prompt's pages
    bd.dflash2_pages_fork(t.pages, i32([0] * samples), i32(list(range(1, rows))), t.kv_len)
    full = lambda v, ty: torch.full((samples,), v, dtype=ty, device="cuda")  # noqa: E731
    temps, ks, tokens = full(temperature, torch.float32), full(top_k, torch.int32), full(0, torch.int32)
    caches, begin = t.caches_of(1, rows), torch.arange(rows, dtype=torch.int32, device="cuda")
    group, prefix = i32([0, samples]), i32([prompt])
    work = torch.empty(bd.dflash2_paged_shared_bytes(t.handle, samples), dtype=torch.uint8, device="cuda")
    logits, new_len, out, most = logits.expand(samples, -1).contiguous(), t.kv_len.clone(), [[] for _ in range(samples)], 0

    def attend(cache, q, o):
        if shared is None:
            bd.dflash2_paged_attention(t.handle, cache, q, o, begin, t.kv_len[1:], max_new=1, max_len=t.max_len, scale=scale)
        else:
            bd.dflash2_paged_attention_shared(t.handle, cache, q, o, begin, t.kv_len[1:], group, prefix, work, max_new=1, max_len=t.max_len,
                                              max_group=samples, max_prefix=prompt, scale=scale, how=shared)

    for i in range(steps):
        if watch is not None:
            watch(logits)
        u = torch.rand(samples, generator=g, device="cuda")
        bd.dflash2_sample(logits, temps, ks, None, None, u, tokens)
        if force is not None:
            tokens.copy_(i32([f[i] for f in force]))
        for o, x in zip(out, tokens.tolist()):
            o.append(x)
        new_len[1:] += 1
        t.resize(new_len)
        most = max(most, int((t.ref > 0).sum()))
        logits = t.forward(caches, tokens, begin, t.kv_len[1:], 1, attend)
    t.resize(torch.zeros_like(new_len))
    assert not t.ref.any()
    t.close()
    return out, most


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--samples", type=int, default=4)
    ap.add_argument("--steps", type=int, default=12)
    ap.add_argument("--temperature", type=float, default=0.9)
    a = ap.parse_args()
    bd.build()
    tokens, pages = run(a.samples, a.steps, temperature=a.temperature)
    for i, t in enumerate(tokens):
        print(f"sample {i}: {t}")
    print(f"{pages} pages held at most")


if __name__ == "__main__":
    main()
