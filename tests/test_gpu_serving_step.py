"""The calls for many samples of one prompt together, as a program runs them."""
import numpy as np
import pytest
import torch

import block_drafter_pos_gb300 as bd
import examples.shared_prompt as ex

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shared", ["together", "apart"])
def test_samples_of_a_prompt_are_plain_decoding(shared):
    """The tokens of samples that share the prompt's pages, judged by the logits of a run whose attention knows nothing of the
    prefix and which is fed the same tokens: at temperature 0 each is that row's best up to near-ties, the outputs that the two
    ways round to bf16 differing in their last bits, 2^-8 each, through two layers (a token of a wrong context is whole standard
    deviations off).  All samples are then the same."""
    got, pages = ex.run(5, 14, temperature=0.0, shared=shared)
    logits = []
    ex.run(5, 14, temperature=0.0, shared=None, force=got, watch=lambda x: logits.append(x.clone()))
    for i, x in enumerate(logits):
        for r, t in enumerate(got):
            assert x[r, t[i]] >= x[r].max() - 2.0 ** -5 * x[r].std(), (i, r)
    # 45 positions of a prompt in pages of 16: two whole pages once, then each row's own
    assert pages == 3 + 5 * 2


def test_samples_go_their_own_ways():
    got, pages = ex.run(4, 9, temperature=1.0)
    assert all(len(t) == 9 for t in got) and len({tuple(t) for t in got}) > 1
    assert pages == 3 + 4 * 2 and all(0 <= x < 4096 for t in got for x in t)


def test_a_trees_accepted_path_is_what_a_chain_writes():
    """The keys and values that a tree's kept nodes leave in the cache (turned by their depths, then moved together) are bit for bit
    those of writing the path as a chain, and the next token's attention gives the same bits.  A token's rows come from a table, so
    that they do not depend on what stands beside them."""
    g = torch.Generator(device="cuda").manual_seed(1)
    row = {n: torch.randn(4096, h, 64, generator=g, device="cuda").to(torch.bfloat16) for n, h in (("q", 8), ("k", 2), ("v", 2))}
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    depth = [0, 1, 1, 2, 2, 3, 3, 4]
    paths = [[0, 2, 4, 5, 7], [0, 1, 3]]
    for page in (16, 5):
        tree, chain = (ex.Target(2, 40, 20, layers=2, page=page, seed=3) for _ in range(2))

        def write(t, tokens, begin, positions=None):
            x = i32(tokens).long()
            for c in t.caches:
                q = row["q"][x]
                bd.dflash2_paged_rope_write(t.handle, t.rope, c, q, q, row["k"][x], row["v"][x], begin, t.kv_len, positions=positions)
            return q

        rng = np.random.default_rng(page)
        nodes = rng.integers(0, 4096, (2, 8)).tolist()
        prompt = rng.integers(0, 4096, 42).tolist()
        for t in (tree, chain):                                               # the prompts, 21 tokens each
            t.resize(i32([21, 21]))
            write(t, prompt, i32([0, 21, 42]))
        tree.resize(i32([29, 29]))
        begin = i32([0, 8, 16])
        write(tree, nodes[0] + nodes[1], begin, i32([21 + d for d in depth] * 2))
        keep, n_keep = torch.zeros(2, 8, dtype=torch.int32, device="cuda"), i32([len(p) for p in paths])
        for r, p in enumerate(paths):
            keep[r, :len(p)] = i32(p)
        new_len = torch.empty_like(tree.kv_len)
        bd.dflash2_paged_keep(tree.handle, tree.caches, begin, tree.kv_len, keep, n_keep, kv_out=new_len)
        assert new_len.tolist() == [26, 24]
        tree.resize(new_len)                                                  # the pages behind the paths go back
        chain.resize(i32([26, 24]))
        write(chain, [nodes[r][i] for r, p in enumerate(paths) for i in p], i32([0, 5, 8]))
        assert tree.ref.tolist() == chain.ref.tolist() and tree.table.tolist() == chain.table.tolist()
        found = []
        for t in (tree, chain):
            t.resize(t.kv_len + 1)
            one = i32([0, 1, 2])
            q = write(t, [7, 9], one)
            for c in t.caches:
                k, v = (torch.zeros(52, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in "kv")
                bd.dflash2_paged_read(t.handle, c, k, v, i32([0, 27, 52]), t.kv_len)
                out = torch.empty_like(q)
                bd.dflash2_paged_attention(t.handle, c, q, out, one, t.kv_len, max_new=1, max_len=t.max_len, scale=0.125)
                found.append((k, v, out))
            t.close()
        for a, b in zip(found[:2], found[2:]):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
            assert bool(a[0].any()) and bool(torch.isfinite(a[2]).all())
