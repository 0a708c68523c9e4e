"""Beams' states follow their parents: arrays in place (tq_states_reorder) and
page tables (tq_pages_reorder) against plain indexing, and beam search over a
paged and a contiguous cache from logits to attention."""
import numpy as np
import pytest
import torch

from _parity import ATTN_ATOL

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def parents(rng, n, W, kind):
    g = np.arange(n).reshape(-1, W)
    if kind == "same":
        p = g
    elif kind == "cycle":
        p = np.roll(g, 1, axis=1)
    elif kind == "one":
        p = np.repeat(g[:, W // 2:W // 2 + 1], W, 1)
    else:
        p = g[:, :1] + rng.integers(0, W, size=g.shape)
    return p.ravel()


def moved(a, parent, lens):
    """The array after every sequence has taken over its parent's slots."""
    b = a.copy()
    W_all = np.arange(len(parent))
    for s in W_all:
        p = parent[s]
        if p == s:
            continue
        n = a.shape[2] if lens is None else min(max(int(lens[p]), 0), a.shape[2])
        b[s, :, :n] = a[p, :, :n]
    return b


@pytest.mark.parametrize("kind", ["random", "cycle", "one", "same"])
@pytest.mark.parametrize("W,groups", [(1, 3), (2, 3), (4, 2), (5, 2), (8, 1), (13, 2), (16, 1), (29, 1), (32, 2), (33, 1), (64, 1)])
def test_states_reorder(tqlib, W, groups, kind):
    """Every column width (rows of 16, 8, 4, 2 and 1 byte multiples), lengths of
    none, some and all slots, the bytes behind them untouched."""
    from turboquant_kv_cache_gb300 import binding as tb
    rng = np.random.default_rng(W)
    n = W * groups
    shapes = [(n, 2, 64, 48), (n, 3, 37, 24), (n, 1, 301, 4), (n, 2, 33, 6), (n, 1, 19, 3), (n, 2, 5, 16), (n, 1, 0, 16), (n, 1, 700, 56)]
    host = [rng.integers(0, 256, size=s, dtype=np.uint8) for s in shapes]
    lens = [rng.integers(-1, s[2] + 3, size=n) for s in shapes]
    lens[5] = None
    lens[0][:] = 64
    lens[2][: n // 2] = 0
    parent = parents(rng, n, W, kind)
    if kind == "random" and W > 1:
        bad = rng.random(n) < 0.1          # parents that are none
        parent = np.where(bad, rng.choice([-1, n, 2**31 - 1, -2**31], n), parent)
        if groups > 1:
            parent[0] = n - 1              # of another group
    arrays = [torch.from_numpy(h).cuda() for h in host]
    states = tb.StateArrays(arrays, [None if x is None else i32(x) for x in lens])
    tb.tq_states_reorder(states, i32(parent), W)
    valid = np.where((parent >= 0) & (parent < n) & (parent // W == np.arange(n) // W), parent, np.arange(n))
    for a, h, x in zip(arrays, host, lens):
        np.testing.assert_array_equal(a.cpu().numpy(), moved(h, valid, x))


def test_states_reorder_caches_and_shapes(tqlib):
    """A packed cache with QJL, an fp16 window, a history; one length tensor for
    all; arrays that start off 16-byte boundaries; replaced arrays followed."""
    from turboquant_kv_cache_gb300 import binding as tb
    W, n, H, cap = 4, 8, 2, 77
    L = tb.make_layout(128, 128, 2, qjl_m=96)
    S = torch.randn(96, 128, device="cuda")
    cache = tb.tq_quantize_kv(L, torch.randn(n, H, cap, 128, device="cuda").half(), S=S)
    win = torch.randn(n, H, cap, 128, device="cuda").half()
    hist = torch.randint(0, 1000, (n * cap + 1,), dtype=torch.int32, device="cuda")[1:].view(n, cap)
    lens = i32([77, 3, 0, 50, 76, 1, 20, 33])
    states = tb.StateArrays([cache, win, hist], lens)
    parent = [1, 0, 3, 3, 7, 4, 5, 6]
    for _ in range(2):
        tensors = [cache.codes, cache.scales, cache.qjl, cache.rnorm, win, hist]
        before = [t.clone() for t in tensors]
        tb.tq_states_reorder(states, i32(parent), W)
        for t, b in zip(tensors, before):
            four = lambda x: x.cpu().numpy().reshape(n, 1 if x.dim() == 2 else H, cap, -1)  # noqa: E731
            np.testing.assert_array_equal(four(t), moved(four(b), np.array(parent), lens.cpu().numpy()))
        states.arrays[1] = win = win.clone()          # another tensor in an entry's place
        cache.codes = cache.codes.clone()
    # the lengths are a state of their own, in a call behind
    tb.tq_states_reorder(tb.StateArrays([lens.view(n, 1)]), i32(parent), W)
    assert lens.tolist() == [3, 77, 50, 50, 33, 76, 1, 20]


def test_copies_know_their_own_arrays(tqlib):
    """Copied and pickled handles follow the copy's arrays, not the first one's."""
    import copy
    import pickle

    from turboquant_kv_cache_gb300 import binding as tb
    a = torch.arange(8, dtype=torch.int32, device="cuda").view(4, 2)
    states = tb.StateArrays([a])
    tb.tq_states_reorder(states, i32([0, 1, 2, 3]), 4)
    for again in (copy.deepcopy(states), pickle.loads(pickle.dumps(states))):
        tb.tq_states_reorder(again, i32([3, 3, 3, 3]), 4)
        assert (again.arrays[0] == a[3]).all() and a.flatten().tolist() == list(range(8))
    slots = tb.tq_batch_slots(i32([1, 1]), None, 2, S_cap=8)
    again = copy.deepcopy(slots)
    tb.tq_batch_slots(i32([2, 0]), None, S_cap=8, out=again)
    assert slots.seq.tolist() == [0, 1] and again.seq.tolist() == [0, 0]


def test_states_reorder_refusals(tqlib):
    from turboquant_kv_cache_gb300 import binding as tb
    a = torch.zeros(8, 2, 16, 4, dtype=torch.uint8, device="cuda")
    n = i32([1] * 8)
    paged = tb.PackedKV(tb.make_layout(64, 64, 4), (8, 2, 32), page_table=i32([[0]] * 8))
    for arrays, lens in (([a, a], None), ([a, a[4:]], None), ([a.transpose(1, 2)], None), ([a], n[:4]), ([a], n.long()), ([], None),
                         ([n.view(8, 1)], n), ([a, a.clone()], [n]), ([a.cpu()], None), ([paged], None), ([n], None)):
        with pytest.raises(ValueError):
            tb.StateArrays(arrays, lens)
    s = tb.StateArrays([a], n)
    for p, W in ((n[:4], 4), (n.long(), 4)):
        with pytest.raises(ValueError):
            tb.tq_states_reorder(s, p, W)
    for W in (0, 3, 65):
        with pytest.raises(tb.TQError):
            tb.tq_states_reorder(s, n, W)


def test_states_reorder_long_rows(tqlib):
    """A row behind 2^31 bytes, a captured replay, another stream."""
    from turboquant_kv_cache_gb300 import binding as tb
    n, H, cap, by = 4, 3, 20_000_003, 16
    a = torch.empty(n, H, cap, by, dtype=torch.uint8, device="cuda")
    for s in range(n):
        a[s].fill_(s + 1)
    lens = i32([cap, cap - 1, 5, cap])
    parent = i32([1, 0, 2, 2])
    states = tb.StateArrays([a], lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    tb.tq_states_reorder(states, parent, 4, stream=side)
    side.synchronize()
    assert (a[0, :, :-1] == 2).all() and (a[0, :, -1] == 1).all() and (a[1] == 1).all() and (a[2] == 3).all()
    assert (a[3, :, :5] == 3).all() and (a[3, :, 5:] == 4).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tb.tq_states_reorder(states, parent, 4)
    graph.replay()
    torch.cuda.synchronize()
    assert (a[0, :, :-1] == 1).all() and (a[1, :, :-1] == 2).all()


def pool_of(rng, n_seqs, pps, shared, spare, W):
    """A pool whose groups of W share their first pages."""
    table = rng.integers(-5, 10**6, size=(n_seqs, pps))   # entries behind the held pages mean nothing
    held = np.zeros(n_seqs, np.int64)
    at, rows = 0, []
    for g in range(0, n_seqs, W):
        prompt = list(range(at, at + shared))
        at += shared
        for s in range(g, min(g + W, n_seqs)):
            m = int(rng.integers(0, pps - shared + 1))
            rows.append(prompt + list(range(at, at + m)))
            if rng.random() < 0.1:
                rows[-1] = []
            at += m
    num = at + spare
    name = rng.permutation(num)
    ref = np.zeros(num, np.int64)
    for s, r in enumerate(rows):
        table[s, :len(r)] = name[r]
        held[s] = len(r)
        ref[name[r]] += 1
    return table, held, ref


@pytest.mark.parametrize("kind", ["random", "cycle", "one", "same"])
@pytest.mark.parametrize("n_seqs,W,pps,shared", [(1, 1, 1, 0), (4, 4, 3, 1), (16, 4, 33, 8), (12, 3, 300, 40), (100, 5, 257, 3),
                                                 (512, 8, 64, 20), (2000, 4, 9, 2)])
def test_pages_reorder(tqlib, n_seqs, W, pps, shared, kind):
    from turboquant_kv_cache_gb300 import binding as tb
    rng = np.random.default_rng(n_seqs + pps)
    table, held, ref = pool_of(rng, n_seqs, pps, shared, 5, W)
    for mode in ("all", "some"):
        pool = tb.PagePool(i32(table), i32(held), i32(ref), 32)
        seqs = None if mode == "all" else rng.permutation(n_seqs)[:max(1, n_seqs * 2 // 3)]
        n = n_seqs if seqs is None else len(seqs)
        if kind == "random" or mode == "some":
            parent = rng.integers(0, n, size=n) if kind != "same" else np.arange(n)
        else:
            parent = parents(rng, n, W, kind)
        ids = np.arange(n) if seqs is None else seqs
        t, h, r = table.copy(), held.copy(), ref.copy()
        for i in range(n):
            np.subtract.at(r, table[ids[i], :held[ids[i]]], 1)
        for i in range(n):
            p = ids[parent[i]]
            t[ids[i], :held[p]] = table[p, :held[p]]
            h[ids[i]] = held[p]
            np.add.at(r, table[p, :held[p]], 1)
        res = tb.tq_pages_reorder(pool, i32(parent), None if seqs is None else i32(seqs))
        assert res.tolist() == [0, int((parent != np.arange(n)).sum()), 0, 0]
        np.testing.assert_array_equal(pool.page_table.cpu().numpy(), t)
        np.testing.assert_array_equal(pool.n_pages.cpu().numpy(), h)
        np.testing.assert_array_equal(pool.ref.cpu().numpy(), r)


@pytest.mark.parametrize("n_seqs,pps", [(8, 40), (96, 300)])
def test_pages_reorder_replayed_and_on_a_stream(tqlib, n_seqs, pps):
    """One workspace for calls in a row; a captured call replayed; another stream."""
    from turboquant_kv_cache_gb300 import binding as tb
    rng = np.random.default_rng(2)
    table, held, ref = pool_of(rng, n_seqs, pps, pps // 3, 5, 4)
    pool = tb.PagePool(i32(table), i32(held), i32(ref), 32)
    ws = torch.empty(tb.tq_pages_reorder_workspace_bytes(n_seqs, pps, n_seqs), dtype=torch.uint8, device="cuda")
    parent = i32(np.arange(n_seqs))
    result = i32([0] * 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    tb.tq_pages_reorder(pool, parent, workspace=ws, result=result, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tb.tq_pages_reorder(pool, parent, workspace=ws, result=result)
        tb.tq_pages_reorder(pool, parent, workspace=ws, result=result)   # the same again
    for _ in range(4):
        p = rng.integers(0, n_seqs, size=n_seqs)
        parent.copy_(i32(p))
        graph.replay()
        for _ in range(2):
            t, h, r = table.copy(), held.copy(), ref.copy()
            for i in range(n_seqs):
                np.subtract.at(r, table[i, :held[i]], 1)
            for i in range(n_seqs):
                t[i, :held[p[i]]] = table[p[i], :held[p[i]]]
                h[i] = held[p[i]]
                np.add.at(r, table[p[i], :held[p[i]]], 1)
            table, held, ref = t, h, r
        torch.cuda.synchronize()
        for got, want in ((pool.page_table, table), (pool.n_pages, held), (pool.ref, ref)):
            np.testing.assert_array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("n_seqs,pps", [(8, 40), (600, 40)])
def test_pages_reorder_refused_entries_change_nothing(tqlib, n_seqs, pps):
    from turboquant_kv_cache_gb300 import binding as tb
    rng = np.random.default_rng(1)
    table, held, ref = pool_of(rng, n_seqs, pps, 4, 5, 4)
    good = rng.integers(0, n_seqs, size=n_seqs)
    for parent, seqs in (((-1, 5), None), ((n_seqs, 5), None), ((0, 1), (2, 2)), ((0, 1), (-1, 2)), ((0, 1), (n_seqs, 2))):
        pool = tb.PagePool(i32(table), i32(held), i32(ref), 32)
        p, s = good.copy(), None
        p[[3, 6]] = parent
        if seqs is not None:
            s = np.arange(n_seqs)
            s[[3, 6]] = seqs
        res = tb.tq_pages_reorder(pool, i32(p), None if s is None else i32(s))
        assert res.tolist() == [-1, 0, 0, 0]
        for got, want in ((pool.page_table, table), (pool.n_pages, held), (pool.ref, ref)):
            np.testing.assert_array_equal(got.cpu().numpy(), want)
    pool = tb.PagePool(i32(table), i32(held), i32(ref), 32)
    assert tb.tq_pages_reorder(pool, i32([])).tolist() == [0, 0, 0, 0]
    for kw in (dict(parent=i32(good).long()), dict(parent=i32(good), seqs=i32(good[:3])), dict(parent=i32(good), result=i32([0])),
               dict(parent=i32(good), workspace=torch.empty(10, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            tb.tq_pages_reorder(pool, **kw)
    with pytest.raises(tb.TQError):
        tb.tq_pages_reorder(pool, i32(list(good) + [0]))


@pytest.mark.parametrize("keep", [True, False])
@pytest.mark.parametrize("d,W,B,page", [(128, 4, 2, 32), (64, 3, 3, 64)])
def test_beam_search_over_paged_and_contiguous_caches(tqlib, d, W, B, page, keep):
    """A search of some steps, its states in pages and, beside them, in a
    contiguous cache with a history: after each step both give the attention of
    every beam's own path of tokens, as a host model follows it, and the pool's
    counts are those of its tables."""
    from turboquant_kv_cache_gb300 import binding as tb
    Hq, Hkv, V, prompt, steps, eos = 4, 2, 501, 45, 9, 3
    n = B * W
    g = torch.Generator(device="cuda").manual_seed(d + W)
    L = tb.make_layout(d, 32, 4)
    pps = (prompt + steps) // page + 2
    num = n * pps + 4
    paged = [tb.PackedKV(L, (num, Hkv, page)) for _ in range(2)]
    cap = prompt + steps
    flat = [tb.PackedKV(L, (n, Hkv, cap)) for _ in range(2)]
    for c in paged + flat:
        c.codes.zero_()
        c.scales.zero_()
    pool = tb.PagePool.new(n, pps, num, page, paged)
    tables = [tb.PackedKV.of(L, c.codes, c.scales, page_table=pool.page_table) for c in paged]
    hist = torch.full((n, cap), -1, dtype=torch.int32, device="cuda")
    # rows of every token at every position of each request, so that a path of tokens gives its keys and values
    rows = torch.randn(2, B, cap, V, Hkv, d, generator=g, device="cuda").half()
    first = i32([b * W for b in range(B)])
    assert tb.tq_pages_fork(pool, i32([-1] * B), first, i32([0] * B), i32([prompt] * B)).tolist()[0] == 0
    start = torch.randint(0, V, (B, prompt), generator=g, device="cuda")
    slots = tb.tq_batch_slots(i32([prompt] * B), None, B * prompt, page_table=pool.page_table[first.long()].contiguous(), page_size=page)
    for i in range(2):
        x = torch.stack([rows[i, b, torch.arange(prompt, device="cuda"), start[b]] for b in range(B)])   # [B, prompt, Hkv, d]
        tb.tq_append_kv_slots(paged[i], x.flatten(0, 1), slots.slot)
        tb.tq_append_kv_slots(flat[i], x.repeat_interleave(W, 0).flatten(0, 1),
                              (torch.arange(n, device="cuda")[:, None] * cap + torch.arange(prompt, device="cuda")).flatten())
    others = [s for s in range(n) if s % W]
    if others:   # the other beams begin as forks of the first, with the prompt's pages
        r = tb.tq_pages_fork(pool, i32([s - s % W for s in others]), i32(others), i32([prompt] * len(others)), i32([prompt] * len(others)))
        assert r.tolist()[0] == 0
    states = tb.StateArrays([*flat, hist], None)
    paths = [start[s // W].tolist() for s in range(n)]
    scores = torch.full((B, W), -float("inf"), device="cuda")
    scores[:, 0] = 0
    done = torch.zeros(B, W, dtype=torch.uint8, device="cuda")
    for step in range(steps):
        at = prompt + step
        logits = 3 * torch.randn(B, W, V, generator=g, device="cuda")
        scores, parent, token, done = tb.tq_beam_select(logits, scores, done=done, eos=eos, keep_place=keep)
        if keep:
            p = parent.view(-1)
            assert (p[p.long()] == p).all()    # who is followed stays
        tb.tq_states_reorder(states, parent.view(-1), W)
        assert tb.tq_pages_reorder(pool, parent.view(-1)).tolist()[0] == 0
        every = i32(range(n))
        assert tb.tq_pages_fork(pool, every, every, i32([at] * n), i32([at + 1] * n)).tolist()[0] == 0
        hist[:, at] = token.view(-1)
        paths = [paths[q] + [t] for q, t in zip(parent.view(-1).tolist(), token.view(-1).tolist())]
        for s in range(n):
            assert hist[s, prompt:at + 1].tolist() == paths[s][prompt:]
        ref = np.zeros(num, np.int64)
        for row, h in zip(pool.page_table.tolist(), pool.n_pages.tolist()):
            assert h == at // page + 1
            np.add.at(ref, row[:h], 1)
        np.testing.assert_array_equal(pool.ref.cpu().numpy(), ref)
        slots = tb.tq_batch_slots(i32([1] * n), i32([at] * n), n, page_table=pool.page_table, page_size=page)
        for i in range(2):
            x = torch.stack([rows[i, s // W, at, paths[s][at]] for s in range(n)])
            tb.tq_append_kv_slots(paged[i], x, slots.slot)
            tb.tq_append_kv_slots(flat[i], x, torch.arange(n, device="cuda") * cap + at)
        q = torch.randn(n, Hq, d, generator=g, device="cuda").half()
        a = tb.tq_decode_attn(*tables, q, kv_len=i32([at + 1] * n))
        b = tb.tq_decode_attn(*flat, q, ctx=at + 1)
        pos = torch.arange(at + 1, device="cuda")
        for s in range(n):
            kv = [tb.tq_dequantize_kv(tb.tq_quantize_kv(L, rows[i, s // W, pos, torch.tensor(paths[s], device="cuda")]),
                                      torch.float32).double().transpose(0, 1).repeat_interleave(Hq // Hkv, 0) for i in range(2)]
            w = torch.einsum("hd,htd->ht", q[s].double(), kv[0]) / d ** 0.5
            want = torch.einsum("ht,htd->hd", w.softmax(-1), kv[1])
            assert (a[s].double() - want).abs().max().item() < ATTN_ATOL, (step, s)
            assert (b[s].double() - want).abs().max().item() < ATTN_ATOL, (step, s)
