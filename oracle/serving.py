"""Oracle of the calls for many samples of one prompt: rotary positions (extended precision), the pages of a pool (one row after
the other), and a tree's kept tokens.  Plain NumPy and Python."""
from __future__ import annotations

import math

import numpy as np


def rope_rates(rot, theta=1e7, scaling="none", factor=1.0, original_len=0, beta_fast=32.0, beta_slow=1.0):
    """Radians per position of each pair, and the amplitude."""
    out = []
    lo = hi = 0.0
    if scaling == "yarn":
        lo, hi = (rot * math.log(original_len / (n * 2 * math.pi)) / (2 * math.log(theta)) for n in (beta_fast, beta_slow))
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rot - 1)
    for i in range(rot // 2):
        f = theta ** (-2 * i / rot)
        if scaling == "linear":
            f /= factor
        elif scaling == "yarn":
            g = min(max((i - lo) / (hi - lo if hi > lo else 0.001), 0.0), 1.0)
            f = f * (1 - g) + f / factor * g
        out.append(f)
    return np.array(out), (0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0)


def rope(x, positions, rates, amplitude=1.0, interleaved=False, inverse=False):
    """Rows x [tokens, heads, dim] turned; and for error bounds, at each turned channel, |a| + |b| of its pair (0 elsewhere)."""
    x = np.asarray(x, np.longdouble)
    half = len(rates)
    turns = np.asarray(positions, np.longdouble)[:, None] * (np.asarray(rates, np.longdouble) / (2 * np.longdouble(np.pi)))
    angle = ((turns - np.rint(turns)).astype(np.float64) * 2 * np.pi)[:, None] * (-1 if inverse else 1)
    c, s = np.cos(angle) * amplitude, np.sin(angle) * amplitude
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    y, reach = x.astype(np.float64), np.zeros(x.shape)
    xa, xb = y[..., a].copy(), y[..., b].copy()
    y[..., a], y[..., b] = xa * c - xb * s, xb * c + xa * s
    reach[..., a] = reach[..., b] = (np.abs(xa) + np.abs(xb)) * amplitude
    return y, reach


# The pages of a pool.  State: table (list of lists), ref (list), kv_len (list).

def pages_resize(table, ref, kv_len, new_len, page):
    """Changes the state; returns copies (a triple per row) and statuses (1: out of bounds, 5: too few free pages)."""
    before, lengths, n, width = list(ref), list(kv_len), len(table), len(table[0])
    pages = lambda t: -(-t // page)  # noqa: E731
    good = [o >= 0 and m >= 0 and pages(o) <= width and pages(m) <= width for o, m in zip(kv_len, new_len)]
    tail = [None] * n
    for r in range(n):
        if good[r] and new_len[r] > kv_len[r] and kv_len[r] % page:
            t = table[r][pages(kv_len[r]) - 1]
            if not 0 <= t < len(ref) or before[t] < 1:
                good[r] = False
            else:
                tail[r] = t
    free = [p for p, h in enumerate(before) if h == 0]
    copies, status, full = [(-1, -1, 0)] * n, [0] * n, False
    # what rows take is settled by what was held before the call; pages are given back before any is taken
    for r in range(n):
        if not good[r]:
            status[r] = 1
        elif new_len[r] <= lengths[r]:
            for c in range(pages(new_len[r]), pages(lengths[r])):
                t = table[r][c]
                table[r][c] = -1
                if 0 <= t < len(ref) and ref[t] > 0:
                    ref[t] -= 1
                else:
                    status[r] = 1
            kv_len[r] = new_len[r]
    for r in range(n):
        old, new = lengths[r], new_len[r]
        if not good[r] or new <= old:
            continue
        have, need = pages(old), pages(new)
        renew = False
        if tail[r] is not None and before[tail[r]] > 1:
            growing = [x for x in range(n) if tail[x] == tail[r]]
            keeper = max(growing, key=lambda x: (lengths[x] % page, -x))   # writes behind what the others hold
            renew = not (len(growing) >= before[tail[r]] and keeper == r)
        want = need - have + renew
        if want and (full or want > len(free)):
            full = True
            status[r] = 5
            continue
        taken, free = free[:want], free[want:]
        for c, p in zip(range(have - renew, need), taken):
            table[r][c] = p
            ref[p] = 1
        if renew:
            copies[r] = (tail[r], taken[0], old % page)
            ref[tail[r]] -= 1
        kv_len[r] = new
    return copies, status


def pages_fork(table, ref, kv_len, parent, child, page):
    """Changes the state; returns statuses."""
    n, width = len(table), len(table[0])
    status = []
    done = []
    for i, (p, c) in enumerate(zip(parent, child)):
        ok = 0 <= p < n and 0 <= c < n and list(child).count(c) == 1 and c not in parent and p not in child
        ok = ok and 0 <= kv_len[p] <= width * page and kv_len[c] == 0
        ok = ok and all(0 <= t < len(ref) for t in table[p][:-(-kv_len[p] // page)])
        status.append(0 if ok else 1)
        if ok:
            done.append((p, c))
    for p, c in done:
        have = -(-kv_len[p] // page)
        table[c][:have] = table[p][:have]
        for t in table[p][:have]:
            ref[t] += 1
        kv_len[c] = kv_len[p]
    return status
