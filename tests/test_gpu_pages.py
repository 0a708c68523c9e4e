"""The page-table calls against a plain sequential model of them: tables,
counts and page contents are equal, refused calls change nothing, and the
books stay right over long random runs."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


class Model:
    """The pool as the calls' documentation has it, entry by entry."""

    def __init__(self, n_seqs, pps, num_pages, page):
        self.table = np.zeros((n_seqs, pps), np.int32)
        self.held = np.zeros(n_seqs, np.int32)
        self.ref = np.zeros(num_pages, np.int32)
        self.data = np.arange(num_pages, dtype=np.int64) + 1000   # what each page holds
        self.page = page

    def fork(self, entries):
        n_seqs, pps = self.table.shape
        kids = [c for _, c, _, _ in entries]
        plan = []
        for p, c, share, new in entries:
            if not (0 <= c < n_seqs and -1 <= p < n_seqs and 0 <= share <= new):
                return [-1, 0, 0, 0]
            if kids.count(c) > 1 or (p >= 0 and p != c and p in kids):
                return [-1, 0, 0, 0]
            held = self.held[p] if p >= 0 else 0
            total = -(-new // self.page)
            if total > pps or share > held * self.page or (p != c and self.held[c]):
                return [-1, 0, 0, 0]
            at, part = divmod(share, self.page)
            if p == c:
                cow = at < held and self.ref[self.table[p, at]] > 1
                places = ([at] if cow else []) + list(range(held, total))
                plan.append((p, c, places, self.table[p, at] if cow and part else -1, self.table[p, at] if cow else -1, 0,
                             max(held, total)))
            else:
                plan.append((p, c, list(range(at, total)), self.table[p, at] if part else -1, -1, at, total))
        free = [int(i) for i in np.flatnonzero(self.ref == 0)]
        need = sum(len(e[2]) for e in plan)
        if need > len(free):
            return [need - len(free), 0, 0, 0]
        copies = []
        for p, c, places, src, drop, shared, total in plan:
            for j in range(shared):
                self.table[c, j] = self.table[p, j]
                self.ref[self.table[c, j]] += 1
            for k, j in enumerate(places):
                self.table[c, j] = free.pop(0)
                self.ref[self.table[c, j]] = 1
                if k == 0 and src >= 0:
                    copies.append((src, self.table[c, j]))
            self.held[c] = total
        for _, _, _, _, drop, _, _ in plan:
            if drop >= 0:
                self.ref[drop] -= 1
        for a, b in copies:
            self.data[b] = self.data[a]
        return [0, need, len(copies), 0]

    def free(self, seqs, keep=None):
        for i, s in enumerate(seqs):
            if not 0 <= s < len(self.held):
                continue
            k = min(-(-max(0, keep[i]) // self.page) if keep is not None else 0, self.table.shape[1])
            for j in range(k, self.held[s]):
                self.ref[self.table[s, j]] -= 1
            self.held[s] = min(self.held[s], k)

    def compact(self):
        live = np.flatnonzero(self.ref > 0)
        holes = [i for i in range(len(live)) if self.ref[i] == 0]
        movers = [int(i) for i in live if i >= len(live)]
        to = {m: h for m, h in zip(movers, holes)}
        for s, n in enumerate(self.held):
            for j in range(n):
                self.table[s, j] = to.get(int(self.table[s, j]), self.table[s, j])
        for m, h in to.items():
            self.ref[h], self.ref[m] = self.ref[m], 0
            self.data[h] = self.data[m]
        return [0, len(live), len(to), 0]


LAYOUTS = {  # (d, block, bits, qjl), Hkv
    "turbo3": ((128, 32, 3, 0), 2), "pervec_d64": ((64, 64, 4, 0), 1), "qjl": ((128, 128, 2, 128), 3),
    "k8": ((64, 32, 8, 0), 2), "d256_1bit": ((256, 256, 1, 0), 5),
}


class Pair:
    """A model and a device pool beside each other."""

    def __init__(self, tb, n_seqs, pps, num_pages, page, names=("turbo3", "turbo3")):
        self.tb, self.m = tb, Model(n_seqs, pps, num_pages, page)
        self.caches = []
        H = LAYOUTS[names[0]][1] if names else 0
        gen = torch.Generator(device="cuda").manual_seed(5)
        for n in names:
            d, block, bits, m = LAYOUTS[n][0]
            c = tb.PackedKV(tb.make_layout(d, block, bits, m), (num_pages, H, page),
                            S=torch.zeros(m, d, device="cuda") if m else None)
            for a in self._arrays(c):
                a.view(torch.uint8).random_(0, 256, generator=gen)
            self.caches.append(c)
        self.first = [[a.clone() for a in self._arrays(c)] for c in self.caches]
        self.pool = tb.PagePool.new(n_seqs, pps, num_pages, page, self.caches)

    @staticmethod
    def _arrays(c):
        return [a for a in (c.codes, c.scales, c.qjl, c.rnorm) if a is not None]

    def i32(self, x):
        return torch.tensor(list(x), dtype=torch.int32, device="cuda")

    def fork(self, entries):
        r = self.tb.tq_pages_fork(self.pool, *(self.i32([e[k] for e in entries]) for k in range(4)))
        want = self.m.fork(entries)
        assert r.tolist() == want
        self.check()
        return want

    def free(self, seqs, keep=None):
        self.tb.tq_pages_free(self.pool, self.i32(seqs), self.i32(keep) if keep is not None else None)
        self.m.free(seqs, keep)
        self.check()

    def compact(self):
        r = self.tb.tq_pages_compact(self.pool)
        assert r.tolist() == self.m.compact()
        self.check()

    def check(self):
        m, p = self.m, self.pool
        assert np.array_equal(p.n_pages.cpu().numpy(), m.held)
        assert np.array_equal(p.ref.cpu().numpy(), m.ref)
        mine = np.arange(m.table.shape[1]) < m.held[:, None]
        assert np.array_equal(p.page_table.cpu().numpy()[mine], m.table[mine])
        # a page of every array holds what it or the page it was copied from held at first
        at = torch.from_numpy(m.data - 1000).cuda()
        for c, first in zip(self.caches, self.first):
            for a, b in zip(self._arrays(c), first):
                assert torch.equal(a.view(torch.uint8), b[at].view(torch.uint8))


def test_begin_fork_grow_free(tqlib):
    from turboquant_kv_cache_gb300 import binding as tb
    p = Pair(tb, 8, 6, 40, 32)
    assert p.fork([(-1, 0, 0, 70), (-1, 3, 0, 1), (-1, 5, 0, 0)]) == [0, 4, 0, 0]
    assert p.fork([(0, 1, 70, 71), (0, 2, 64, 64), (0, 4, 64, 65), (0, 6, 0, 40)]) == [0, 1 + 0 + 1 + 2, 1, 0]
    assert p.fork([(0, 0, 70, 100), (1, 1, 70, 70), (3, 3, 1, 1)]) == [0, 1, 0, 0]
    # sequence 2 rolls back into a page it shares, then writes: it gets its own copy
    p.free([2], [40])
    assert p.fork([(2, 2, 40, 41)]) == [0, 1, 1, 0]
    # at a page's start there is nothing to copy, only a page of its own to take
    p.free([4], [64])
    assert p.fork([(4, 4, 32, 33)]) == [0, 1, 0, 0]
    p.free([0, 1])
    p.compact()
    p.free(range(8))
    assert not p.pool.ref.any()
    p.compact()


def test_two_owners_of_a_page_both_replace_it(tqlib):
    from turboquant_kv_cache_gb300 import binding as tb
    p = Pair(tb, 4, 4, 16, 32)
    p.fork([(-1, 0, 0, 64)])
    p.fork([(0, 1, 64, 64)])
    assert p.fork([(0, 0, 50, 51), (1, 1, 50, 51)]) == [0, 2, 2, 0]
    assert p.pool.ref[1].item() == 0


@pytest.mark.parametrize("entries,status", [
    ([(0, 1, 33, 33), (0, 1, 33, 33)], -1),          # a child named twice
    ([(0, 1, 33, 33), (1, 2, 0, 0)], -1),            # a parent that is a child
    ([(0, 0, 60, 70), (0, 1, 10, 10)], -1),          # a parent that grows
    ([(0, 3, 10, 10)], -1),                          # a child that holds pages
    ([(0, 1, 97, 97)], -1),                          # more than the parent has
    ([(0, 1, 20, 10)], -1),                          # less than it shares
    ([(0, 1, -1, 10)], -1), ([(-1, 1, 1, 10)], -1), ([(-2, 1, 0, 10)], -1), ([(9, 1, 0, 10)], -1), ([(0, 8, 0, 10)], -1),
    ([(0, -1, 0, 10)], -1), ([(-1, 1, 0, 6 * 32 + 1)], -1),
    ([(-1, 1, 0, 5 * 32), (-1, 2, 0, 2 * 32)], 1),   # six free pages
    ([(-1, 1, 0, 6 * 32), (-1, 2, 0, 6 * 32), (-1, 4, 0, 1)], 7),
])
def test_refused_entries_change_nothing(tqlib, entries, status):
    from turboquant_kv_cache_gb300 import binding as tb
    p = Pair(tb, 8, 6, 10, 32)
    p.fork([(-1, 0, 0, 96), (-1, 3, 0, 5)])
    assert p.fork(entries)[0] == status
    assert p.fork([(0, 7, 33, 34)]) == [0, 1, 1, 0]   # and the pool is as good as before


@pytest.mark.parametrize("names", [(), ("turbo3",), ("qjl", "qjl"), ("k8", "turbo3"), ("d256_1bit",), ("pervec_d64",) * 70])
def test_layouts_and_many_caches(tqlib, names):
    """Every array of every cache moves; more arrays than one launch takes."""
    from turboquant_kv_cache_gb300 import binding as tb
    p = Pair(tb, 6, 8, 30, 32, names)
    p.fork([(-1, 0, 0, 100), (-1, 1, 0, 40), (-1, 2, 0, 200)])
    p.fork([(0, 3, 99, 100), (2, 4, 161, 161), (1, 5, 3, 3)])
    p.free([0, 1])
    p.compact()


def test_free_twice_out_of_range_and_longer_than_held(tqlib):
    from turboquant_kv_cache_gb300 import binding as tb
    p = Pair(tb, 6, 8, 64, 32)
    p.fork([(-1, i, 0, 32 * (i + 1)) for i in range(6)])
    p.fork([])
    p.free([5, 5, -1, 6, 1000, 4], [64, 32, 0, 0, 0, 10000])
    p.free([])
    p.free([3, 3, 3, 2], [-5, 96, 64, 33])
    p.free([0, 0])


@pytest.mark.parametrize("n_seqs,pps,num_pages,page,steps", [(9, 7, 40, 32, 60), (64, 40, 1500, 64, 25),
                                                              (300, 12, 2049, 32, 20), (1300, 5, 5000, 32, 6),
                                                              (40, 30, 17000, 32, 8), (420, 48, 2500, 32, 8),
                                                              (1300, 90, 6000, 32, 4)])
def test_random_runs(tqlib, n_seqs, pps, num_pages, page, steps):
    """Random steps of a scheduler, more sequences and pages than a block
    takes at once, until the pool is short; pools on both sides of the size
    that one block serves."""
    from turboquant_kv_cache_gb300 import binding as tb
    p = Pair(tb, n_seqs, pps, num_pages, page, ("pervec_d64",))
    rng = np.random.default_rng(n_seqs)
    length = np.zeros(n_seqs, np.int64)
    short = 0
    for step in range(steps):
        busy = [int(s) for s in np.flatnonzero(p.m.held)]
        idle = [int(s) for s in np.flatnonzero(p.m.held == 0)]
        rng.shuffle(busy)
        rng.shuffle(idle)
        n_kid = int(rng.integers(0, min(len(idle), 1 + n_seqs // 3) + 1))
        parents, grows = busy[:len(busy) // 2], busy[len(busy) // 2:]
        entries = []
        for c in idle[:n_kid]:
            if parents and rng.random() < 0.7:
                par = parents[int(rng.integers(0, min(3, len(parents))))]
                share = int(rng.integers(0, length[par] + 1))
                entries.append((par, c, share, min(pps * page, share + int(rng.integers(0, 2 * page)))))
            else:
                entries.append((-1, c, 0, int(rng.integers(0, pps * page + 1))))
        for g in grows[:int(rng.integers(0, len(grows) + 1))]:
            entries.append((g, g, int(length[g]), min(pps * page, int(length[g] + rng.integers(0, page)))))
        order = [entries[i] for i in rng.permutation(len(entries))]
        if p.fork(order)[0] == 0:
            for par, c, share, new in order:
                length[c] = new
        else:
            short += 1
        busy = [int(s) for s in np.flatnonzero(p.m.held)]
        gone = [s for s in busy if rng.random() < (0.6 if short and step % 3 == 0 else 0.2)]
        keep = [int(rng.integers(0, length[s] + 1)) if rng.random() < 0.4 else 0 for s in gone]
        p.free(gone, keep)
        for s, k in zip(gone, keep):
            length[s] = min(length[s], k)
        if step % 4 == 3:
            p.compact()


def test_table_entries_that_are_no_page(tqlib):
    """A table that names no page where a copy is due is refused; one in a
    full page's place is passed on without a count; nothing is read or
    written outside the arrays, and compaction leaves such entries."""
    from turboquant_kv_cache_gb300 import binding as tb
    p = Pair(tb, 4, 4, 8, 32)
    p.fork([(-1, 0, 0, 96)])
    before = [t.clone() for t in (p.pool.page_table, p.pool.n_pages, p.pool.ref)]
    for bad in (-1, 8, 1 << 30, -(1 << 31)):
        p.pool.page_table[0, 1] = bad
        r = tb.tq_pages_fork(p.pool, p.i32([0]), p.i32([1]), p.i32([33]), p.i32([33]))
        assert r.tolist() == [-1, 0, 0, 0]
        r = tb.tq_pages_fork(p.pool, p.i32([0]), p.i32([1]), p.i32([64]), p.i32([64]))
        assert r.tolist() == [0, 0, 0, 0] and p.pool.page_table[1, 1].item() == bad
        tb.tq_pages_compact(p.pool)
        assert p.pool.page_table[1, 1].item() == bad
        tb.tq_pages_free(p.pool, p.i32([1]))
        for a, b in zip((p.pool.page_table, p.pool.n_pages, p.pool.ref), before):
            a.copy_(b)
    p.check()
    # a table that names a free page behind the pages in use
    p.pool.page_table[0, 2] = 7
    tb.tq_pages_compact(p.pool)
    assert p.pool.page_table[0, :3].tolist() == [0, 1, 7]


def test_captured_replay(tqlib):
    """A captured free, fork and compaction replayed on a changed pool."""
    from turboquant_kv_cache_gb300 import binding as tb
    p = Pair(tb, 8, 6, 40, 32)
    p.fork([(-1, 0, 0, 70), (-1, 1, 0, 100)])
    done, par, kid, share, new = (p.i32(x) for x in ([1], [0], [2], [70], [72]))
    res, res2 = p.i32([9] * 4), p.i32([9] * 4)
    ws = torch.empty(tb.tq_pages_workspace_bytes(8, 40, 1), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tb.tq_pages_free(p.pool, done)
        tb.tq_pages_fork(p.pool, par, kid, share, new, workspace=ws, result=res)
        tb.tq_pages_compact(p.pool, workspace=ws, result=res2)
    for d, e in ((1, (0, 2, 70, 72)), (0, (2, 4, 33, 97)), (7, (4, 5, 90, 91)), (7, (4, 5, 90, 91))):
        for t, x in zip((done, par, kid, share, new), (d,) + e):
            t.fill_(x)
        g.replay()
        p.m.free([d])
        assert res.tolist() == p.m.fork([e])
        assert res2.tolist() == p.m.compact()
        p.check()


def test_binding_refusals(tqlib):
    from turboquant_kv_cache_gb300 import binding as tb
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    with pytest.raises(ValueError):
        tb.PagePool(z(4, 8), z(3), z(10), 32)
    with pytest.raises(ValueError):
        tb.PagePool(z(4, 8), z(4), z(10).long(), 32)
    L = tb.make_layout(64, 32, 4)
    with pytest.raises(ValueError):
        tb.PagePool(z(4, 8), z(4), z(10), 32, [tb.PackedKV(L, (9, 2, 32))])
    with pytest.raises(ValueError):
        tb.PagePool(z(4, 8), z(4), z(10), 32, [tb.PackedKV(L, (10, 2, 32)), tb.PackedKV(L, (10, 1, 32))])
    pool = tb.PagePool(z(4, 8), z(4), z(10), 32)
    with pytest.raises(ValueError):
        tb.tq_pages_fork(pool, z(2), z(1), z(1), z(1))
    with pytest.raises(tb.TQError):
        tb.tq_pages_fork(pool, z(5), z(5), z(5), z(5))
    with pytest.raises(ValueError):
        tb.tq_pages_free(pool, z(2), z(1))


def test_replaced_arrays_are_followed(tqlib):
    """The page calls work on the pool's and the caches' arrays as they are at
    the call, and refuse what no longer fits."""
    from turboquant_kv_cache_gb300 import binding as tb
    L = tb.make_layout(64, 32, 4)
    c = tb.PackedKV(L, (20, 2, 32))
    c.codes.view(-1).copy_(torch.arange(c.codes.numel(), device="cuda") % 251)
    c.scales.fill_(1)
    pool = tb.PagePool.new(4, 6, 20, 32, [c])
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    fork = lambda *e: tb.tq_pages_fork(pool, *(i32(x) for x in e)).tolist()  # noqa: E731
    assert fork(-1, 0, 0, 40) == [0, 2, 0, 0]
    old = c.codes
    c.codes = old.clone()
    first = old.clone()
    assert fork(0, 1, 40, 40) == [0, 1, 1, 0]                      # page 1 copied to page 2, in the new array
    assert torch.equal(old, first)
    assert torch.equal(c.codes[2], first[1]) and torch.equal(c.codes[3:], first[3:])
    # a wider table, other books
    was = pool.page_table, pool.n_pages, pool.ref
    pool.page_table = torch.zeros(4, 9, dtype=torch.int32, device="cuda")
    pool.page_table[:, :6] = was[0]
    pool.ref, pool.n_pages = was[2].clone(), was[1].clone()
    kept = [t.clone() for t in was]
    assert fork(1, 1, 40, 9 * 32) == [0, 7, 0, 0] and pool.n_pages.tolist() == [2, 9, 0, 0]
    assert all(torch.equal(a, b) for a, b in zip(was, kept))
    tb.tq_pages_free(pool, i32(0))
    assert tb.tq_pages_compact(pool).tolist() == [0, 9, 1, 0]
    assert torch.equal(c.codes[1], first[9]) and torch.equal(old, first)
    # a table of the same storage with other rows
    pool.page_table = pool.page_table.view(-1)[:32].view(4, 8)
    assert pool.books() and pool.struct.pages_per_seq == 8
    # what no longer fits is refused before anything runs
    c.codes = old[:19].contiguous()
    for call in (lambda: fork(-1, 2, 0, 1), lambda: tb.tq_pages_compact(pool)):
        with pytest.raises(ValueError):
            call()
    c.codes = old
    pool.n_pages = pool.n_pages[:3].clone()
    for call in (lambda: fork(-1, 2, 0, 1), lambda: tb.tq_pages_compact(pool), lambda: tb.tq_pages_free(pool, i32(0))):
        with pytest.raises(ValueError):
            call()
    pool.n_pages, pool.ref = was[1].clone(), was[2].long()
    with pytest.raises(ValueError):
        tb.tq_pages_free(pool, i32(0))
