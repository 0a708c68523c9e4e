"""Ragged batches: the place of every row (tq_batch_slots) against a loop over
the sequences, and rows quantised into their slots (tq_append_kv_slots) against
tq_quantize_kv of the same rows, whose codes are tested against the oracle."""
import numpy as np
import pytest
import torch

from _parity import ATTN_ATOL

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def layout_of(new, have, n_rows, cap, table=None, page=0):
    """Rows of the batch one by one."""
    start, seq, pos, slot = [0], [], [], []
    for b, (n, h) in enumerate(zip(new, have)):
        for j in range(n):
            p = h + j
            seq.append(b)
            pos.append(p)
            slot.append(b * cap + p if table is None else int(table[b][p // page]) * page + p % page)
        start.append(len(seq))
    k = n_rows - len(seq)
    rows = None if table is None else np.array([table[b] for b in seq] + [[0] * len(table[0])] * k, np.int32).reshape(n_rows, len(table[0]))
    return dict(row_start=start, seq=seq + [-1] * k, pos=pos + [-1] * k, slot=slot + [-1] * k,
                row_len=[p + 1 for p in pos] + [0] * k, row_table=rows)


def check(out, ref, status=0):
    assert out.result.tolist() == [status, ref["row_start"][-1] if status == 0 else 0, 0, 0]
    for name, want in ref.items():
        got = getattr(out, name)
        if got is not None:
            np.testing.assert_array_equal(got.cpu().numpy(), np.asarray(want, dtype=got.cpu().numpy().dtype), err_msg=name)


@pytest.mark.parametrize("B,n_rows,page,pps", [
    (1, 1, 32, 1), (1, 0, 32, 2), (3, 7, 32, 5), (5, 131, 96, 3), (8, 96, 32, 64), (300, 4099, 64, 33), (1025, 9001, 32, 3),
    (2048, 9001, 32, 3), (2049, 9001, 32, 3), (4096, 9001, 32, 3), (4097, 9001, 32, 3), (9000, 20003, 32, 2), (17, 5000, 0, 0), (5000, 70001, 0, 0)])
def test_batch_slots(tqlib, B, n_rows, page, pps):
    from turboquant_kv_cache_gb300 import binding as tb
    rng = np.random.default_rng(B + n_rows)
    cap = page * pps or 700
    new = np.where(rng.random(B) < 0.3, 0, rng.integers(0, 1 + min(cap, 2 * n_rows // B), size=B))
    while new.sum() > n_rows:
        new = new * 3 // 4
    if n_rows > B:
        new[-1] = min(cap, n_rows - new[:-1].sum())   # mostly a full buffer
    have = (rng.random(B) * (cap - new + 1)).astype(np.int64)
    table = rng.permutation(B * pps).reshape(B, pps) if page else None
    out = tb.tq_batch_slots(i32(new), i32(have), n_rows, S_cap=cap, page_table=i32(table) if page else None, page_size=page,
                            row_table=bool(page) and n_rows < 10000)
    check(out, layout_of(new, have, n_rows, cap, table, page))


@pytest.mark.parametrize("B", [3, 5000])
def test_batch_slots_statuses_and_defaults(tqlib, B):
    """Too many rows, lengths that are not valid, no cached tokens; outputs
    given and used again; a part of a wider table."""
    from turboquant_kv_cache_gb300 import binding as tb
    rng = np.random.default_rng(B)
    new = rng.integers(0, 4, size=B)
    total, pps, page = int(new.sum()), 4, 32
    wide = i32(rng.permutation(B * 7).reshape(B, 7))
    table = wide[:, 2:6]
    host = table.cpu().numpy()
    out = tb.BatchSlots.new(B, total, row_pages=pps)
    tb.tq_batch_slots(i32(new), None, page_table=table, page_size=page, out=out)
    check(out, layout_of(new, [0] * B, total, pps * page, host, page))
    none = layout_of([0] * B, [0] * B, total, pps * page, host, page)
    more = new.copy()
    more[1] += 5
    tb.tq_batch_slots(i32(more), None, page_table=table, page_size=page, out=out)
    check(out, none, status=5)
    have = np.zeros(B, np.int64)
    for bad_new, bad_have in ((-1, 0), (1, -1), (1, pps * page), (2**31 - 1, 1), (pps * page + 1, 0)):
        m, h = new.copy(), have.copy()
        m[-1], h[-1] = bad_new, bad_have
        tb.tq_batch_slots(i32(m), i32(h), page_table=table, page_size=page, out=out)
        check(out, none, status=-1)
    huge = np.full(B, 2**31 - 200)   # the sum passes 32 bits
    r = tb.tq_batch_slots(i32(huge), None, total, S_cap=2**31 - 100)
    assert r.result.tolist()[0] == min(int(huge.sum()) - total, 2**31 - 1) and not r.row_start.any() and (r.slot == -1).all()
    t2 = i32(host)
    t2[0] = -1   # a sequence whose pages are gone
    out = tb.tq_batch_slots(i32(new), None, total, page_table=t2, page_size=page)
    assert (out.slot[out.seq == 0] == -1).all() and (out.slot[out.seq > 0] >= 0).all()


def test_batch_slots_least_outputs_on_a_stream(tqlib):
    """Only what has to be there, new lengths that start off 16 bytes, a stream."""
    from turboquant_kv_cache_gb300 import binding as tb
    lens = i32([9, 2, 0, 5, 1])
    e = lambda n, dt=torch.int32: torch.empty(n, dtype=dt, device="cuda")  # noqa: E731
    out = tb.BatchSlots(e(5), None, e(9), e(9, torch.int64), None, None, None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    tb.tq_batch_slots(lens[1:], None, S_cap=16, out=out, stream=side)
    new = tb.tq_batch_slots(lens[1:], lens[1:], 9, S_cap=16, stream=side)
    side.synchronize()
    ref = layout_of([2, 0, 5, 1], [0] * 4, 9, 16)
    for name in ("row_start", "pos", "slot"):
        assert getattr(out, name).tolist() == ref[name]
    check(new, layout_of([2, 0, 5, 1], [2, 0, 5, 1], 9, 16))


def test_batch_slots_refusals(tqlib):
    from turboquant_kv_cache_gb300 import binding as tb
    n, t = i32([1, 2]), i32([[0, 1], [2, 3]])
    for kw in (dict(n_rows=4), dict(S_cap=64), dict(n_rows=4, page_table=t, page_size=32, S_cap=65),
               dict(n_rows=4, page_table=t.long(), page_size=32), dict(n_rows=4, page_table=t[:1], page_size=32),
               dict(n_rows=4, page_table=t.t(), page_size=32), dict(out=tb.BatchSlots.new(3, 4), S_cap=64),
               dict(out=tb.BatchSlots.new(2, 4), S_cap=64, n_rows=5),
               dict(out=tb.BatchSlots.new(2, 4, row_pages=3), page_table=t, page_size=32)):
        with pytest.raises(ValueError):
            tb.tq_batch_slots(n, None, **kw)
    with pytest.raises(ValueError):
        tb.tq_batch_slots(n, i32([1]), 4, S_cap=64)
    with pytest.raises(tb.TQError):
        tb.tq_batch_slots(n, None, 4, page_table=t, page_size=33)


LAYOUTS = [  # head_dim, block, bits, qjl, norm_correct, fp32 input: over the quantise kernels
    (128, 32, 3, 0, 0, False), (64, 64, 4, 0, 0, False), (256, 32, 4, 0, 0, False), (128, 128, 2, 128, 0, False),
    (256, 64, 3, 0, 0, False), (128, 128, 2, 64, 1, False), (64, 64, 1, 0, 0, True), (128, 32, 8, 0, 0, False), (256, 256, 3, 0, 1, True)]


@pytest.mark.parametrize("page", [0, 32, 96])
@pytest.mark.parametrize("d,block,bits,m,nc,f32", LAYOUTS)
def test_append_slots(tqlib, d, block, bits, m, nc, f32, page):
    """Records equal to tq_quantize_kv's, in their slots; every other slot, and
    those of rows without one, untouched."""
    from turboquant_kv_cache_gb300 import binding as tb
    rng = np.random.default_rng(d + bits + page)
    L = tb.make_layout(d, block, bits, qjl_m=m, norm_correct=nc)
    S = torch.from_numpy(rng.standard_normal((m, d)).astype(np.float32)).cuda() if m else None
    for n, H in ((1, 1), (7, 3), (301, 2)):
        lead = (n // 16 + 3, H, page or 37)
        n_slots = lead[0] * lead[2]
        slot = rng.permutation(n_slots)[:n].astype(np.int64)
        slot[rng.random(n) < 0.2] = -1
        if n > 3:
            slot[1], slot[3] = n_slots, 1 << 40   # outside the cache
        x = torch.from_numpy(rng.standard_normal((n, H, d)).astype(np.float32)).cuda()
        x = x if f32 else x.half()
        cache = tb.PackedKV(L, lead, S=S)
        arrays = [t for t in (cache.codes, cache.scales, cache.qjl, cache.rnorm) if t is not None]
        for t in arrays:
            t.view(torch.uint8).fill_(0xA5)
        before = [t.clone() for t in arrays]
        want = tb.tq_quantize_kv(L, x, S=S)
        assert tb.tq_append_kv_slots(cache, x, torch.from_numpy(slot).cuda()) is cache
        fine = np.nonzero((slot >= 0) & (slot < n_slots))[0]
        page_of, off = slot[fine] // lead[2], slot[fine] % lead[2]
        for t, b, w in zip(arrays, before, (want.codes, want.scales, want.qjl, want.rnorm)):
            b[torch.from_numpy(page_of).cuda(), :, torch.from_numpy(off).cuda()] = w[torch.from_numpy(fine).cuda()]
            assert torch.equal(t.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("d,block,bits,H,n", [(64, 64, 4, 1, 700001), (128, 32, 3, 3, 300001), (64, 32, 2, 8, 90001)])
def test_append_slots_many_rows(tqlib, d, block, bits, H, n):
    """Rows on both sides of what a block keeps the records of; the last rows of
    a batch and of a block."""
    from turboquant_kv_cache_gb300 import binding as tb
    L = tb.make_layout(d, block, bits)
    page = 64
    pages = n // page + 2
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randn(n, H, d, generator=g, device="cuda").half()
    slot = torch.randperm(pages * page, generator=g, device="cuda")[:n]
    slot[::13] = -1
    cache = tb.PackedKV(L, (pages, H, page))
    cache.codes.zero_()
    cache.scales.zero_()
    tb.tq_append_kv_slots(cache, x, slot)
    want = tb.tq_quantize_kv(L, x)
    for got, rows in ((cache.codes, want.codes), (cache.scales, want.scales)):
        live = slot >= 0
        ref = torch.zeros_like(got)
        ref[slot[live] // page, :, slot[live] % page] = rows[live]
        assert torch.equal(got.view(torch.uint8), ref.view(torch.uint8))


def test_append_slots_refusals(tqlib):
    from turboquant_kv_cache_gb300 import binding as tb
    cache = tb.PackedKV(tb.make_layout(64, 64, 4), (2, 3, 32))
    x, slot = torch.zeros(5, 3, 64, device="cuda"), torch.zeros(5, dtype=torch.int64, device="cuda")
    for bad_x, bad_slot in ((x[:, :2], slot), (x[:4], slot), (x, slot.int()), (x[..., :32], slot), (x[None], slot), (x, slot.cpu()),
                            (x.transpose(0, 1), slot), (x.cpu(), slot)):
        with pytest.raises(ValueError):
            tb.tq_append_kv_slots(cache, bad_x, bad_slot)
    with pytest.raises(TypeError):
        tb.tq_append_kv_slots(cache, x.double(), slot)
    tb.tq_append_kv_slots(cache, x[:0], slot[:0])


@pytest.mark.parametrize("d,page,Hq,Hkv", [(128, 32, 8, 2), (64, 64, 4, 4)])
def test_ragged_batch_end_to_end(tqlib, d, page, Hq, Hkv):
    """Prompts of unequal lengths packed in one buffer: slots, norm and rotation
    by row (each row a batch entry of one token), append, and every row's
    attention over its own table row, captured and replayed with other lengths."""
    from turboquant_kv_cache_gb300 import binding as tb
    B, n_rows, pps = 5, 24, 4
    rng = np.random.default_rng(d)
    L = tb.make_layout(d, 32, 4)
    caches = [tb.PackedKV(L, (B * pps + 2, Hkv, page)) for _ in range(2)]
    for c in caches:
        c.codes.zero_()
        c.scales.zero_()
    table = i32(rng.permutation(B * pps + 2)[:B * pps].reshape(B, pps))
    cap = pps * page
    ang = np.arange(cap)[:, None] * 1e4 ** (-np.arange(0, d, 2) / d)
    rope = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).cuda()
    w = torch.ones(d, device="cuda")
    new, have = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    qkv = torch.zeros(n_rows, 1, (Hq + 2 * Hkv) * d, device="cuda")
    slots = tb.BatchSlots.new(B, n_rows, row_pages=pps)
    pages = [tb.PackedKV.of(L, c.codes, c.scales, page_table=slots.row_table) for c in caches]
    state = {}

    def step():
        tb.tq_batch_slots(new, have, page_table=table, page_size=page, out=slots)
        q, k, v = tb.tq_qkv_norm_rope(qkv, Hq, Hkv, d, w, w, rope=rope, pos=slots.pos)
        for c, x in zip(caches, (k, v)):
            tb.tq_append_kv_slots(c, x[:, :, 0], slots.slot)
        q = q[:, :, 0].contiguous()
        state["q"], state["out"] = q, tb.tq_decode_attn(*pages, q, kv_len=slots.row_len)

    step()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    lens = np.zeros(B, np.int64)
    for rows in ([7, 0, 9, 1, 5], [1, 1, 1, 1, 1], [0, 20, 0, 2, 1], [0, 0, 0, 0, 0]):
        new.copy_(i32(rows))
        have.copy_(i32(lens))
        qkv.copy_(torch.from_numpy(rng.standard_normal(qkv.shape).astype(np.float32)))
        graph.replay()
        torch.cuda.synchronize()
        check(slots, layout_of(rows, lens, n_rows, cap, table.cpu().numpy(), page))
        deq = [tb.tq_dequantize_kv(c, torch.float32).double() for c in caches]
        r = 0
        for b in range(B):
            kk, vv = (x[table[b].long()].transpose(0, 1).flatten(1, 2).repeat_interleave(Hq // Hkv, 0) for x in deq)
            for j in range(rows[b]):
                n = lens[b] + j + 1
                s = torch.einsum("hd,htd->ht", state["q"][r].double(), kk[:, :n]) / d ** 0.5
                ref = torch.einsum("ht,htd->hd", s.softmax(-1), vv[:, :n])
                assert (state["out"][r].double() - ref).abs().max().item() < ATTN_ATOL
                r += 1
        assert not state["out"][r:].any()
        lens += rows


def test_append_slots_stream_and_offsets(tqlib):
    """A call on another stream, and records behind 2^31 bytes of codes."""
    from turboquant_kv_cache_gb300 import binding as tb
    L = tb.make_layout(256, 32, 4)
    n_pages, H, page = 40000, 8, 64    # 2.6 GB of codes
    cache = tb.PackedKV(L, (n_pages, H, page))
    cache.codes[-1].zero_()
    x = torch.randn(6, H, 256, device="cuda").half()
    slot = torch.tensor([n_pages * page - 1, n_pages * page - 64, 5, n_pages * page, -5, 2**62], device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    tb.tq_append_kv_slots(cache, x, slot, stream=s)
    s.synchronize()
    want = tb.tq_quantize_kv(L, x)
    assert torch.equal(cache.codes[-1, :, 63], want.codes[0]) and torch.equal(cache.codes[-1, :, 0], want.codes[1])
    assert torch.equal(cache.codes[0, :, 5], want.codes[2]) and not cache.codes[-1, :, 1:63].any()
