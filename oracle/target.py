"""FP64 oracle of the target's side of a step: the cache's quantisation, attention of new
tokens over a cache, and truncated sampling.  Plain NumPy, one request or row at a time."""
from __future__ import annotations

import numpy as np

QMAX = {"int8": 127.0, "e4m3": 448.0}


def e4m3_round(y):
    """y rounded to the nearest value of the 8-bit format with 4 exponent and 3 mantissa bits
    (ties to even, saturating at 448): steps of 2^(e - 3) in [2^e, 2^(e + 1)), e >= -6."""
    y = np.asarray(y, np.float64)
    a = np.abs(y)
    e = np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -6.0)
    step = np.exp2(e - 3)
    return np.sign(y) * np.minimum(np.rint(a / step) * step, 448.0)


def quantise(x, fmt):
    """(values of the codes, scales) of rows x [..., D]: scale = max(amax / Q, 2^-126) and code =
    x / scale in FP32, rounded to nearest.  A row that is not finite gets zero codes and a nonfinite scale."""
    x = np.asarray(x, np.float32)
    q = np.float32(QMAX[fmt])
    with np.errstate(all="ignore"):
        amax = np.max(np.abs(x), axis=-1)
        scale = (amax / q).astype(np.float32)
        ok = np.isfinite(amax)
        scale = np.where(ok, np.maximum(scale, np.float32(2.0 ** -126)), scale).astype(np.float32)
        y = np.where(ok[..., None], x / scale[..., None], np.float32(0)).astype(np.float32)
    codes = np.clip(np.rint(y.astype(np.float64)), -127, 127) if fmt == "int8" else e4m3_round(y)
    return codes, scale


def visible(n, length, causal=True, window=0, tree=None):
    """[n, length] truth values: what new token i (position length - n + i) sees."""
    p = length - n + np.arange(n)[:, None]
    j = np.arange(length)[None, :]
    see = np.ones((n, length), bool)
    if tree is not None:
        rel = j - (length - n)
        bits = (np.asarray(tree, np.uint64)[:, None] >> np.clip(rel, 0, 63).astype(np.uint64)) & np.uint64(1)
        see &= (rel < 0) | (bits == 1)
    elif causal:
        see &= j <= p
    if window > 0:
        see &= p - j < window
    return see


def paged_attention(q, k, v, scale, see):
    """q [n, Hq, D], k, v [length, Hkv, D], see [n, length] -> out [n, Hq, D], lse [n, Hq], and for
    error bounds spread = sum_j w_j |v_j| [n, Hq, D] and reach = max_j scale sum_d |q_d k_jd| [n, Hq]."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    n, hq, d = q.shape
    g = hq // k.shape[1]
    out, lse = np.zeros((n, hq, d)), np.full((n, hq), -np.inf)
    spread, reach = np.zeros((n, hq, d)), np.zeros((n, hq))
    for i in range(n):
        js = np.nonzero(see[i])[0]
        if len(js) == 0:
            continue
        for h in range(hq):
            kk, vv = k[js, h // g], v[js, h // g]
            with np.errstate(all="ignore"):
                s = kk @ q[i, h] * scale
                m = s.max()
                e = np.exp(s - m)
                l = e.sum()
                out[i, h] = (e[:, None] * vv).sum(0) / l
                lse[i, h] = m + np.log(l)
                spread[i, h] = (e[:, None] * np.abs(vv)).sum(0) / l
                reach[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(scale)
    return out, lse, spread, reach


def truncated_sample(x, temperature, top_k, top_p, min_p, u):
    """One row of logits -> (token, probability, stays [V], margin): margin is the smallest distance, in
    shares of the weight concerned, of any decision from its border (infinite where none is near)."""
    token, prob, stays, cut, draw = truncated_sample_margins(x, temperature, top_k, top_p, min_p, u)
    return token, prob, stays, min(cut, draw)


def truncated_sample_margins(x, temperature, top_k, top_p, min_p, u):
    """The same with two margins: of what stays, and of the draw.  Decisions without a rounding have none: the largest
    logit's weight is 1; where every weight is 1 or too small to count, sums are whole numbers; and at u = 0 ids whose running
    weight is 0 are passed over."""
    x = np.asarray(x, np.float64)
    order = np.argsort(-x, kind="stable")            # logit descending, id ascending
    v = len(x)
    cut = draw = np.inf
    if temperature == 0:
        stays = np.zeros(v, bool)
        stays[order[0]] = True
        return int(order[0]), 1.0, stays, cut, draw
    xs = x[order]
    w = np.exp((xs - xs[0]) / float(temperature))
    n = top_k if 0 < top_k < v else v
    w[n:] = 0.0
    whole = ((w == 1.0) | (w < 2.0 ** -80)).all()
    if whole:
        w = np.where(w == 1.0, 1.0, 0.0)
    keep = np.arange(v) < n
    if top_p < 1:
        total, run = w.sum(), np.cumsum(w)
        before = np.concatenate([[0.0], run[:-1]])
        keep &= (before < float(top_p) * total) | (np.arange(v) == 0)
        if not whole:
            cut = min(cut, np.abs(run - float(top_p) * total).min() / total)
    if min_p > 0:
        cut = min(cut, np.abs(w[keep & (w < 1.0)] - float(min_p)).min(initial=np.inf))
        keep &= w >= float(min_p)
    keep &= xs > -np.inf
    stays = np.zeros(v, bool)
    stays[order[keep]] = True
    mass = np.zeros(v)
    mass[order] = np.where(keep, w, 0.0)
    cdf = np.cumsum(mass)
    goal = float(u) * cdf[-1]
    token = int(np.searchsorted(cdf, goal, side="right"))
    if not whole:
        draw = np.abs(cdf[cdf > 0.0] - goal).min() / cdf[-1]
    return token, mass[token] / cdf[-1], stays, cut, draw
