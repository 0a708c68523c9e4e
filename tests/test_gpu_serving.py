"""The serving calls together, as a server runs them: a prompt is normalised,
rotated and appended to pages, samples fork from it, each step's rows are
appended to their own pages and attend to the shared prefix and their own
tokens, some end, the pool is compacted, and the rest goes on.  Every step is
checked against attention in 64 bits over the decoded rows."""
import math

import numpy as np
import pytest
import torch

from turboquant_kv_cache_gb300 import inputs

from _parity import ATTN_ATOL

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,kbits,Hq,Hkv,page,prompt", [(128, 3, 8, 2, 32, 130), (64, 4, 4, 2, 64, 129), (256, 4, 8, 2, 32, 64)])
def test_fork_norm_append_attend_free_compact(tqlib, d, kbits, Hq, Hkv, page, prompt):
    from turboquant_kv_cache_gb300 import binding as tb
    n_seqs, pps, num_pages, steps = 8, 16, 96, 12
    L = tb.make_layout(d, 32, kbits)
    caches = [tb.PackedKV(L, (num_pages, Hkv, page)) for _ in range(2)]
    for c in caches:
        c.codes.zero_()
        c.scales.zero_()
    pool = tb.PagePool.new(n_seqs, pps, num_pages, page, caches)
    i32 = lambda x: torch.tensor(list(x), dtype=torch.int32, device="cuda")  # noqa: E731
    view = lambda c, t: tb.PackedKV.of(L, c.codes, c.scales, page_table=t)  # noqa: E731
    ang = np.arange(600)[:, None] * 1e4 ** (-np.arange(0, d, 2) / d)
    rope = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).cuda()
    w = torch.ones(d, device="cuda")
    norm = lambda x, pos: tb.tq_qkv_norm_rope(x, Hq, Hkv, d, w, w, rope=rope, pos=pos)  # noqa: E731
    rows = lambda B, T, seed: torch.from_numpy(inputs.gaussian((B, T, (Hq + 2 * Hkv) * d), seed)).cuda()  # noqa: E731

    # the prompt, in sequence 0, and some short-lived sequences around it
    assert tb.tq_pages_fork(pool, i32([-1, -1]), i32([6, 7]), i32([0, 0]), i32([3 * page, page])).tolist()[0] == 0
    assert tb.tq_pages_fork(pool, i32([-1]), i32([0]), i32([0]), i32([prompt])).tolist()[0] == 0
    q, k, v = norm(rows(1, prompt, 1), i32([0]))
    for c, x in zip(caches, (k, v)):
        tb.tq_append_kv(view(c, pool.page_table[:1]), x, i32([0]))
    dead = i32([6, 7])
    tb.tq_pages_free(pool, dead)

    # samples 1..4 fork from it: whole pages shared, the part-filled one copied
    live = [1, 2, 3, 4]
    shared = prompt // page          # pages that all of them hold
    r = tb.tq_pages_fork(pool, i32([0] * 4), i32(live), i32([prompt] * 4), i32([prompt + 1] * 4)).tolist()
    assert r == [0, 4, 4 if prompt % page else 0, 0]
    tb.tq_pages_free(pool, i32([0]))   # the samples keep the prompt's pages alive
    n = prompt
    for step in range(steps):
        if step == 5:
            tb.tq_pages_free(pool, i32([2]))
            live = [1, 3, 4]
        if step in (3, 6, 9):
            res = tb.tq_pages_compact(pool).tolist()
            assert res[1] == int((pool.ref > 0).sum()) and not pool.ref[res[1]:].any()
        B = len(live)
        ids = i32(live)
        if step:
            r = tb.tq_pages_fork(pool, ids, ids, i32([n] * B), i32([n + 1] * B)).tolist()
            assert r[0] == 0 and r[2] == 0
        table = pool.page_table[ids.long()].contiguous()
        q, k, v = norm(rows(B, 1, 100 + step), i32([n] * B))
        K, V = (view(c, table) for c in caches)
        for c, x in zip((K, V), (k, v)):
            tb.tq_append_kv(c, x, i32([n] * B))
        n += 1
        q = q[:, :, 0].contiguous()
        own = table[:, shared:]
        out = tb.tq_decode_attn_shared(*(view(c, table[:1, :shared]) for c in caches), *(view(c, own) for c in caches), q,
                                       prefix_ctx=shared * page, ctx=own.shape[1] * page,
                                       kv_len=i32([n - shared * page] * B))
        plain = tb.tq_decode_attn(K, V, q, ctx=n)
        deq = [tb.tq_dequantize_kv(c, torch.float32).double() for c in caches]
        for b in range(B):
            kk, vv = (x[table[b].long()].transpose(0, 1).flatten(1, 2)[:, :n].repeat_interleave(Hq // Hkv, 0) for x in deq)
            s = torch.einsum("hd,htd->ht", q[b].double(), kk) / math.sqrt(d)
            ref = torch.einsum("ht,htd->hd", s.softmax(-1), vv)
            assert (out[b].double() - ref).abs().max().item() < ATTN_ATOL, step
            assert (plain[b].double() - ref).abs().max().item() < ATTN_ATOL, step
    tb.tq_pages_free(pool, i32(live))
    assert not pool.ref.any() and not pool.n_pages.any()
