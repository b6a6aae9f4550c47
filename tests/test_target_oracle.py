"""The sampling oracle's margins: which of its decisions a rounding could turn."""
import numpy as np

from oracle import target as ot


def test_exact_decisions_have_no_margin():
    inf = np.inf
    x = np.zeros(50)
    for k, p, m, u in [(0, 1.0, 1.0, 0.0), (7, 0.5, 1.0, 0.25), (0, 0.5, 0.0, 0.5), (49, 1.0, 1.0, 1 - 2.0 ** -24)]:
        tok, prob, stays, cut, draw = ot.truncated_sample_margins(x, 0.7, k, p, m, u)
        n = int(np.ceil((k or 50) * p))
        assert cut == draw == inf and stays.sum() == n and stays[:n].all() and prob == 1 / n
        assert tok == int(np.floor(u * n))
    x[:] = -300.0
    x[[3, 30]] = 1.0                                           # the others' weights are nothing
    tok, prob, stays, cut, draw = ot.truncated_sample_margins(x, 1.0, 0, 0.5, 0.0, 0.0)
    assert cut == draw == inf and tok == 3 and prob == 1.0 and stays.sum() == 1
    # the largest against min_p = 1, and ids cut before the first that stays at u = 0, among weights that are rounded
    x = np.linspace(0.0, 3.0, 50)
    tok, prob, stays, cut, draw = ot.truncated_sample_margins(x, 1.0, 0, 1.0, 1.0, 0.0)
    assert tok == 49 and stays.sum() == 1 and cut > 0.05 and draw == 1.0
    tok, _, _, cut, draw = ot.truncated_sample_margins(x, 1.0, 5, 1.0, 0.0, 0.0)
    assert tok == 45 and cut == inf and draw > 0.1


def test_rounded_decisions_have_one():
    x = np.log(np.array([4.0, 2.0, 1.0, 1.0]))
    _, _, stays, cut, _ = ot.truncated_sample_margins(x, 1.0, 0, 0.5 + 2.0 ** -40, 0.0, 0.9)
    assert stays.sum() == 2 and 0 < cut < 2.0 ** -38
    _, _, _, cut, _ = ot.truncated_sample_margins(x, 1.0, 0, 1.0, 0.5 - 2.0 ** -40, 0.9)
    assert 0 < cut < 2.0 ** -38
    tok, _, _, cut, draw = ot.truncated_sample_margins(x, 1.0, 0, 1.0, 0.0, 0.75 - 2.0 ** -40)
    assert tok == 1 and cut == np.inf and 0 < draw < 2.0 ** -38
    assert ot.truncated_sample(x, 1.0, 0, 1.0, 0.0, 0.75 - 2.0 ** -40)[3] == draw
