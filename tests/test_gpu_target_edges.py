"""Places where the target's side of a step can go wrong."""

import numpy as np
import pytest
import torch

from test_gpu_target import Setup

pytestmark = pytest.mark.gpu

# ----------------------------------------------------------------------------- what a row does not see

@pytest.mark.parametrize("fmt", ["bf16", "fp16"])
def test_nonfinite_values_in_many_small_units(fmt):
    """Units of one and of two row tiles after one another in a CTA, nonfinite values in some of them."""
    g = np.random.default_rng(4)
    new = [int(n) for n in g.choice([20, 40], 700)]            # 80 or 160 rows per KV head
    s = Setup(new, new, hq=8, hk=2, dim=64, page=16, fmt=fmt, seed=9)
    q = s.queries(fmt)
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
