"""What the pages' calls are for: no position that a row holds is written by another row.  A model of the pages' contents that
knows nothing of how pages are chosen: every position carries a tag, copies are applied as noted, and rows write what they grew by."""
import numpy as np
import pytest
import torch

import block_drafter_pos_gb300 as bd
from oracle import serving as os_


class Oracle:
    """The calls as the oracle makes them."""

    def __init__(self, rows, width, n_pages, page):
        self.state, self.page = ([[-1] * width for _ in range(rows)], [0] * n_pages, [0] * rows), page

    def resize(self, new):
        return os_.pages_resize(*self.state, new, self.page)

    def fork(self, parent, child):
        return os_.pages_fork(*self.state, parent, child, self.page)

    def look(self):
        return self.state


class Device:
    """The calls as the library makes them."""

    def __init__(self, rows, width, n_pages, page):
        i32 = lambda *s, v=0: torch.full(s, v, dtype=torch.int32, device="cuda")  # noqa: E731
        self.table, self.ref, self.kv, self.copies = i32(rows, width, v=-1), i32(n_pages), i32(rows), i32(3, rows)
        self.pool = bd.page_pool(self.table, self.ref, page)

    def _on(self, a):
        return torch.tensor(a, dtype=torch.int32, device="cuda")

    def resize(self, new):
        status = torch.zeros_like(self.kv)
        bd.dflash2_pages_resize(self.pool, self.kv, self._on(new), self.copies, status)
        return [tuple(c) for c in self.copies.T.tolist()], status.tolist()

    def fork(self, parent, child):
        status = self._on([0] * len(parent))
        bd.dflash2_pages_fork(self.pool, self._on(parent), self._on(child), self.kv, status)
        return status.tolist()

    def look(self):
        return self.table.tolist(), self.ref.tolist(), self.kv.tolist()


class Contents:
    def __init__(self, make, rows, width, n_pages, page):
        self.calls, self.page, self.step = make(rows, width, n_pages, page), page, 0
        self.pages = [[None] * page for _ in range(n_pages)]
        self.rows = [[] for _ in range(rows)]              # the tags that each row holds

    def check(self):
        table, ref, kv = self.calls.look()
        held = [0] * len(ref)
        for r, tags in enumerate(self.rows):
            assert kv[r] == len(tags)
            assert [self.pages[table[r][x // self.page]][x % self.page] for x in range(len(tags))] == tags, f"row {r}"
            for p in table[r][:-(-len(tags) // self.page)]:
                held[p] += 1
        assert held == ref

    def resize(self, new):
        self.step += 1
        copies, status = self.calls.resize(new)
        table, _, kv = self.calls.look()
        before = [list(p) for p in self.pages]
        for src, dst, n in copies:
            if src >= 0:
                self.pages[dst][:n] = before[src][:n]
        for r, tags in enumerate(self.rows):
            assert status[r] in (0, 5) and kv[r] == (len(tags) if status[r] else new[r])
            for x in range(len(tags), kv[r]):
                tags.append((r, x, self.step))
                self.pages[table[r][x // self.page]][x % self.page] = tags[-1]
            del tags[kv[r]:]
        self.check()
        return status

    def fork(self, parent, child):
        assert self.calls.fork(parent, child) == [0] * len(parent)
        for p, c in zip(parent, child):
            self.rows[c] = list(self.rows[p])
        self.check()


MAKERS = [Oracle, pytest.param(Device, marks=pytest.mark.gpu)]


@pytest.mark.parametrize("make", MAKERS)
@pytest.mark.parametrize("lengths", [[10, 13], [13, 10], [12, 12], [1, 15, 8], [8, 1, 15], [15, 15, 1]])
def test_a_holder_that_is_not_served_keeps_what_it_holds(make, lengths):
    """Sharers of a page, some of them cut, all grow where no page is left: what the page's keeper writes next is nobody's."""
    n = len(lengths)
    c = Contents(make, n + 1, 3, 1, 16)
    c.resize([15] + [0] * n)
    c.fork([0] * n, list(range(1, n + 1)))
    c.resize([0] + lengths)                                # (the first is done)
    status = c.resize([0] + [x + 1 for x in lengths])
    longest = 1 + lengths.index(max(lengths))
    assert [s == 0 for s in status] == [r in (0, longest) for r in range(n + 1)]
    c.resize([len(t) if r != longest else 16 for r, t in enumerate(c.rows)])       # (the page's last position)
    c.resize([len(t) if r != longest else 0 for r, t in enumerate(c.rows)])
    c.resize([0] * (n + 1))


@pytest.mark.parametrize("make", MAKERS)
@pytest.mark.parametrize("rows,width,n_pages,page,seed", [(4, 3, 6, 16, 0), (6, 4, 10, 7, 1), (9, 3, 12, 24, 2), (16, 2, 20, 16, 3), (40, 3, 45, 5, 4)])
def test_no_row_writes_what_another_holds(make, rows, width, n_pages, page, seed):
    """Rows are forked, sharers cut a little, all grow, some are freed, at random and in a pool that runs short."""
    g = np.random.default_rng(seed)
    c = Contents(make, rows, width, n_pages, page)
    met = 0                                                # pages whose holders differ, all ask for more, and some are not served
    lengths = lambda: np.array([len(t) for t in c.rows])  # noqa: E731
    for _ in range(20):
        kv = lengths()
        start = np.where((kv == 0) & (g.random(rows) < 0.3), g.integers(1, 2 * page, rows), kv)
        c.resize(start.tolist())
        kv = lengths()
        free = [int(x) for x in np.nonzero(kv == 0)[0][:3]]
        if free and (kv > 0).any():
            parent = int(g.choice(np.nonzero(kv > 0)[0]))
            c.fork([parent] * len(free), free)
            kv = lengths()
            c.resize([max(int(kv[r]) - int(g.integers(0, 4)), 0) if r in free + [parent] else int(kv[r]) for r in range(rows)])
            kv = lengths()
        new = np.where(kv > 0, np.minimum(kv + g.integers(1, page + 2, rows), width * page), 0)
        table, ref, _ = c.calls.look()
        share = {}
        for r in range(rows):
            if kv[r] % page:
                share.setdefault(table[r][int(kv[r]) // page], []).append(r)
        status = c.resize(new.tolist())
        met += sum(len(rs) == ref[p] and len({int(kv[r]) for r in rs}) > 1 and all(new[r] > kv[r] for r in rs) and any(status[r] for r in rs)
                   for p, rs in share.items())
        kv = lengths()
        c.resize(np.where(g.random(rows) < 0.4, 0, kv).tolist())
    assert met > 0
    c.resize([0] * rows)


@pytest.mark.gpu
@pytest.mark.parametrize("cut", [0, 4])
@pytest.mark.parametrize("rows", [2, 9, 200])
def test_a_page_that_a_row_does_not_hold_is_not_given_back_under_its_new_holder(rows, cut):
    """The first half's tables name free pages (of no holder); they are cut, and so flagged, while the second half takes those
    pages: every taken page has its one holder."""
    half, page = rows // 2, 4
    d = Device(rows, 4, 8 * rows, page)
    d.table[:half, :2] = torch.arange(2 * half, dtype=torch.int32, device="cuda").view(half, 2)
    d.kv[:half] = 8
    for _ in range(3):
        copies, status = d.resize([cut] * half + [11] * (rows - half))
        table, ref, kv = d.look()
        assert status == [1] * half + [0] * (rows - half) and kv == [cut] * half + [11] * (rows - half)
        taken = [t for row in table[half:] for t in row[:3]]
        assert taken == list(range(3 * (rows - half))) and [t for t, h in enumerate(ref) if h] == taken and set(ref) <= {0, 1}
        assert all(t == -1 for row in table[:half] for t in row[-(-cut // page):])
        # as before: the taken pages given back, the first half's tables broken again
        d.resize([cut] * half + [0] * (rows - half))
        d.table[:half, :2] = torch.arange(2 * half, dtype=torch.int32, device="cuda").view(half, 2)
        d.kv[:half] = 8
