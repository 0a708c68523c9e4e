"""Growing a sequence that holds shared pages behind the one its next token
goes to: every page that a token goes to becomes its own."""
import numpy as np
import pytest
import torch

from test_gpu_pages import Model, Pair

pytestmark = pytest.mark.gpu


class TailModel(Model):
    """The model with the rule for a growing sequence's pages in full."""

    def fork(self, entries):
        lost = {}    # entry -> the pages behind its first that it replaces
        for i, (p, c, share, new) in enumerate(entries):
            if p == c and 0 <= c < len(self.held) and 0 <= share <= new:
                at, total = share // self.page, -(-new // self.page)
                row = self.table[c]
                lost[i] = [j for j in range(at, min(self.held[c], max(total, at + 1))) if self.ref[row[j]] > 1]
        self.lost = lost
        return self._fork(entries)

    def _fork(self, entries):
        # the base class's steps with its plan's places and drops in full
        n_seqs, pps = self.table.shape
        kids = [c for _, c, _, _ in entries]
        plan = []
        for i, (p, c, share, new) in enumerate(entries):
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
                lost = self.lost[i]
                plan.append((p, c, lost + list(range(held, total)), self.table[p, at] if part and at in lost else -1,
                             [self.table[p, j] for j in lost], 0, max(held, total)))
            else:
                plan.append((p, c, list(range(at, total)), self.table[p, at] if part else -1, [], at, total))
        free = [int(i) for i in np.flatnonzero(self.ref == 0)]
        need = sum(len(e[2]) for e in plan)
        if need > len(free):
            return [need - len(free), 0, 0, 0]
        copies = []
        for p, c, places, src, drops, shared, total in plan:
            for j in range(shared):
                self.table[c, j] = self.table[p, j]
                self.ref[self.table[c, j]] += 1
            for k, j in enumerate(places):
                self.table[c, j] = free.pop(0)
                self.ref[self.table[c, j]] = 1
                if k == 0 and src >= 0:
                    copies.append((src, self.table[c, j]))
            self.held[c] = total
        for e in plan:
            for page in e[4]:
                self.ref[page] -= 1
        for a, b in copies:
            self.data[b] = self.data[a]
        return [0, need, len(copies), 0]


def _pair(tb, *args):
    p = Pair(tb, *args)
    m = TailModel(*args[:4])
    p.m = m
    return p


@pytest.mark.parametrize("pages", [20, 17000])   # one block, and a pool beyond it
def test_rolled_back_sequence_gets_the_pages_it_writes(tqlib, pages):
    """B forks from A, A rolls back to 40 tokens without giving pages up and
    grows to 128 again: no page that its tokens 40 to 127 go to is B's."""
    from turboquant_kv_cache_gb300 import binding as tb
    p = _pair(tb, 4, 6, pages, 32, ("pervec_d64",))
    p.fork([(-1, 0, 0, 128)])
    p.fork([(0, 1, 128, 128)])
    before = p.pool.page_table[1, :4].clone()
    assert p.fork([(0, 0, 40, 128)]) == [0, 3, 1, 0]
    assert torch.equal(p.pool.page_table[1, :4], before)
    assert p.pool.page_table[0, 0] == before[0] and p.pool.ref[before.long()].tolist() == [2, 1, 1, 1]
    assert not set(p.pool.page_table[0, 1:4].tolist()) & set(before.tolist())
    # up to new_len only: sequence 1 keeps its last page shared with 2, and grows past what it holds
    p.fork([(1, 2, 128, 128)])
    assert p.fork([(1, 1, 32, 70)]) == [0, 2, 0, 0]
    assert p.pool.page_table[1, 3] == p.pool.page_table[2, 3]
    assert p.fork([(2, 2, 65, 192)]) == [0, 3, 0, 0]      # its own third page, the shared last one, two more
    # two owners roll back over the same pages
    p.free([0, 1, 2])
    p.fork([(-1, 0, 0, 160)])
    p.fork([(0, 1, 160, 160), (0, 2, 64, 64)])
    assert p.fork([(0, 0, 33, 150), (1, 1, 10, 100)]) == [0, 4 + 4, 2, 0]
    # short of pages: nothing changes
    if pages == 20:
        p.fork([(1, 3, 160, 160)])
        assert p.fork([(2, 2, 64, 192)]) == [0, 4, 0, 0]
        assert p.fork([(1, 1, 0, 192)]) == [1, 0, 0, 0]   # six pages due; 20 less 11 held and 4 are free


@pytest.mark.parametrize("n_seqs,pps,num_pages,page,steps", [(9, 70, 400, 32, 40), (64, 100, 4000, 32, 10),
                                                              (40, 120, 17000, 32, 8), (1100, 8, 6000, 32, 4)])
def test_random_roll_backs(tqlib, n_seqs, pps, num_pages, page, steps):
    """Sequences that fork, roll back to any length and grow from there, with
    ranges of one page and of more than a warp looks at at once."""
    from turboquant_kv_cache_gb300 import binding as tb
    p = _pair(tb, n_seqs, pps, num_pages, page, ("pervec_d64",))
    rng = np.random.default_rng(pps)
    length = np.zeros(n_seqs, np.int64)
    replaced = 0
    for step in range(steps):
        busy = [int(s) for s in np.flatnonzero(p.m.held)]
        idle = [int(s) for s in np.flatnonzero(p.m.held == 0)]
        rng.shuffle(busy)
        rng.shuffle(idle)
        parents, grows = busy[:len(busy) // 2], busy[len(busy) // 2:]
        entries = []
        for c in idle[:1 + len(idle) // 3]:
            if parents and rng.random() < 0.8:
                par = parents[int(rng.integers(0, min(3, len(parents))))]
                share = int(rng.integers(length[par] // 2, length[par] + 1))
                entries.append((par, c, share, share))
            else:
                entries.append((-1, c, 0, int(rng.integers(0, pps * page + 1))))
        for g in grows:
            share = int(rng.integers(0, length[g] + 1))
            entries.append((g, g, share, int(rng.integers(share, pps * page + 1))))
        order = [entries[i] for i in rng.permutation(len(entries))]
        if p.fork(order)[0] == 0:
            replaced += sum(len(x) for x in p.m.lost.values())
            for _, c, _, new in order:
                length[c] = new
        for s in [s for s in range(n_seqs) if p.m.held[s]]:
            if rng.random() < 0.4:
                p.free([s])
                length[s] = 0
    assert replaced > steps


@pytest.mark.parametrize("num_pages,n_seqs,pps", [(4000, 6, 2300), (8000, 6, 2300), (17000, 6, 4200), (4000, 200, 700), (9000, 1100, 20)])
def test_long_rows_and_many_sequences(tqlib, num_pages, n_seqs, pps):
    """Rows longer than a block takes at once, shared, rolled back over and
    compacted; pools, entries and sequences on both sides of what one block
    takes."""
    from turboquant_kv_cache_gb300 import binding as tb
    p = _pair(tb, n_seqs, pps, num_pages, 32, ("pervec_d64",))
    held = min(pps - 3, num_pages // 2)
    assert p.fork([(-1, 1, 0, 40), (-1, 0, 0, held * 32 - 5)])[0] == 0
    assert p.fork([(0, c, held * 32 - 5 - c % 27, held * 32 - 5 - c % 27) for c in range(2, n_seqs)])[0] == 0
    p.free([1])
    p.compact()
    assert p.fork([(2, 2, held * 16 + 3, held * 32 + 40)])[0] == 0       # half of the row replaced
    p.free([0])
    p.compact()
    p.free([c for c in range(3, n_seqs)])
    p.compact()
