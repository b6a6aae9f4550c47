"""The target's side together with the drafter's: the example's loop, and truncated target rows in the verify."""
import dataclasses

import numpy as np
import pytest
import torch

import block_drafter_pos_gb300 as bd
import examples.target_step as ex
import workloads as wk
from oracle import target as ot

pytestmark = pytest.mark.gpu


def test_greedy_steps_are_plain_decoding():
    """At temperature 0 every token that the verified blocks emit is the argmax of decoding one token at a time
    over the same tokens, up to near-ties: the activations that the two ways round to bf16 and int8 differ in
    their last bits, 2^-8 each, through two layers; a token of a wrong context is whole standard deviations off."""
    greedy = ex.Settings(temperature=0.0)
    got, mean = ex.run(6, greedy)
    assert mean >= 1
    n = min(len(t) for t in got) - 1
    logits = []
    ex.run(n, greedy, plain=True, force=got, watch=lambda x: logits.append(x.cpu()))
    for i, x in enumerate(logits):
        for r, t in enumerate(got):
            assert x[r, t[i + 1]] >= x[r].max() - 2.0 ** -5 * x[r].std(), (i, r)


def test_sampled_steps_run():
    got, mean = ex.run(5, ex.Settings(0.9, 30, 0.9, 0.01))
    assert 1 <= mean <= 8 and all(len(t) >= 6 and all(0 <= x < wk.TOY.vocab for x in t) for t in got)


def test_truncated_rows_bound_what_verify_emits():
    """Rows of dflash2_sample's `kept` as the target of dflash2_verify: every token it emits stays under the
    truncation of its row, a proposal that was cut is rejected, and the emitted probabilities are those of the
    truncated distribution."""
    g = dataclasses.replace(wk.TOY, vocab=8192)
    W = wk.make_weights(g, "bf16", 3)
    R, B, P = 4, 8, 7
    rng = np.random.default_rng(5)
    d = bd.Drafter(g, "bf16", W, R, 256)
    z = torch.from_numpy(rng.normal(0, 2.0, (R * B, g.vocab)).astype(np.float32)).cuda()
    T = 0.8
    vec = lambda v, n, t: torch.full((n,), v, dtype=t, device="cuda")  # noqa: E731
    kept = torch.empty_like(z)
    bd.dflash2_sample(z, vec(T, R * B, torch.float32), vec(25, R * B, torch.int32), vec(0.9, R * B, torch.float32), None,
                      vec(0.5, R * B, torch.float32), torch.empty(R * B, dtype=torch.int32, device="cuda"), kept=kept)
    stays = [ot.truncated_sample(z[i].double().cpu().numpy(), float(np.float32(T)), 25, float(np.float32(0.9)), 0.0, 0.5)[2]
             for i in range(R * B)]
    assert all(np.array_equal(kept[i].cpu().numpy() > -1e29, stays[i]) for i in range(R * B))
    # proposals: the row's best token, but a cut one at position r of request r
    best = z.view(R, B, -1).argmax(-1).to(torch.int32)
    path = best[:, :P].contiguous()
    for r in range(R):
        path[r, r] = int(np.nonzero(~stays[r * B + r])[0][0])
    ids = torch.zeros(R, P, 16, dtype=torch.int32, device="cuda")
    ids[:, :, 0] = path
    ids[:, :, 1:] = torch.arange(1, 16, device="cuda") + 4000
    q = torch.zeros(R, P, 16, device="cuda")
    q[:, :, 0] = 1e-6                                       # so that a token that stays is always accepted
    q[:, :, 1] = 1 - 1e-6
    temps = vec(T, R, torch.float32)
    out, n_acc, n_out = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((R, B), (R,), (R,)))
    probs, status = torch.zeros(R, B, 2, device="cuda"), torch.zeros(R, dtype=torch.int32, device="cuda")
    for seed in range(20):
        seeds, offs = vec(seed, R, torch.int64), torch.arange(R, dtype=torch.int64, device="cuda")
        bd.dflash2_verify(d.handle, R, kept, path, ids, q, temps, seeds, offs, n_acc, out, n_out, probs, status)
        assert not status.any()
        for r in range(R):
            assert int(n_acc[r]) == r and int(n_out[r]) == r + 1
            for i, tok in enumerate(out[r, :r + 1].tolist()):
                assert stays[r * B + i][tok]
    d.close()
