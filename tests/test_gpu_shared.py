"""tq_decode_attn_shared: one softmax over a prefix that all sequences share
and each sequence's own tokens, against attention in 64 bits over the decoded
vectors (the oracle's own packed bytes in one case), on every layout family,
group size and cache form, with empty parts, odd lengths and captured
replays."""
import math

import numpy as np
import pytest
import torch

from oracle import tq_oracle as O
from turboquant_kv_cache_gb300 import inputs

from _parity import ATTN_ATOL, to_np, upload_packed

pytestmark = pytest.mark.gpu


def _cache(tb, L, lead, seed, S=None, scale=1.0):
    x = torch.from_numpy(inputs.gaussian(lead + (L.head_dim,), seed, np.float32) * scale).cuda()
    return tb.tq_quantize_kv(L, x.half(), S=S)


def _reference(tb, Kp, Vp, P, K, V, lens, q, scale=None):
    """Attention of q over the decoded prefix and own tokens, in 64 bits."""
    B, Hq, d = q.shape
    dec = lambda c: tb.tq_dequantize_kv(c, torch.float32).double()  # noqa: E731
    kp, vp = dec(Kp)[0], dec(Vp)[0]
    ko, vo = (dec(K), dec(V)) if K is not None else (None, None)
    G = Hq // kp.shape[0]
    out = torch.zeros(B, Hq, d, dtype=torch.float64, device=q.device)
    for b in range(B):
        for h in range(Hq):
            k, v = kp[h // G, :P], vp[h // G, :P]
            if ko is not None:
                k, v = torch.cat([k, ko[b, h // G, :lens[b]]]), torch.cat([v, vo[b, h // G, :lens[b]]])
            if k.shape[0]:
                s = (k @ q[b, h].double()) * (scale or 1 / math.sqrt(d))
                out[b, h] = torch.softmax(s, 0) @ v
    return out


def _paged(tb, C, page, seed, extra=2, table=None):
    """The cache scattered into shuffled pages, its tail rows zeroed (K and V
    of a call share their table)."""
    B, H, cap = C.lead_shape
    pps = -(-cap // page)
    perm = np.random.default_rng(seed).permutation(B * pps + extra)[:B * pps].reshape(B, pps).astype(np.int32)
    P = tb.PackedKV(C.layout, (B * pps + extra, H, page), S=C.S,
                    page_table=torch.from_numpy(perm).cuda() if table is None else table)
    for name in ("codes", "scales", "qjl", "rnorm"):
        src, dst = getattr(C, name), getattr(P, name)
        if src is None:
            continue
        dst.zero_()
        for b in range(B):
            for j in range(pps):
                n = min(page, cap - j * page)
                dst[int(perm[b, j]), :, :n] = src[b, :, j * page:j * page + n]
    return P


CASES = [
    # name, d, K (block, bits, m, nc), V, B, Hq, Hkv, P_cap, prefix, cap, ctx, lens
    ("turbo3_gqa4", 128, (32, 3, 0, 0), (32, 3, 0, 0), 5, 32, 8, 640, 600, 96, 90, [90, 0, 1, 33, 64]),
    ("turbo3_one_sequence", 128, (32, 3, 0, 0), (32, 3, 0, 0), 1, 8, 2, 1000, 999, 64, 31, [31]),
    ("turbo3_rows_127", 128, (32, 3, 0, 0), (32, 3, 0, 0), 127, 2, 2, 321, 321, 40, 40, None),
    ("turbo3_rows_128", 128, (32, 3, 0, 0), (32, 3, 0, 0), 32, 8, 2, 300, 257, 32, 32, None),
    ("turbo3_rows_132", 128, (32, 3, 0, 0), (32, 3, 0, 0), 33, 8, 2, 300, 256, 32, 7, None),
    ("turbo3_rows_264", 128, (32, 3, 0, 0), (32, 3, 0, 0), 33, 16, 2, 520, 513, 32, 7, None),
    ("prefix_one_token", 128, (32, 3, 0, 0), (32, 3, 0, 0), 3, 8, 2, 1, 1, 64, 64, [64, 0, 5]),
    ("prefix_63", 128, (32, 4, 0, 0), (32, 3, 0, 0), 3, 8, 2, 64, 63, 64, 0, None),
    ("no_prefix", 128, (32, 3, 0, 0), (32, 3, 0, 0), 3, 8, 2, 64, 0, 64, 60, [60, 0, 5]),
    ("no_tokens", 128, (32, 3, 0, 0), (32, 3, 0, 0), 3, 8, 2, 64, 0, 64, 0, None),
    ("prefix_only_long", 128, (32, 2, 0, 0), (32, 3, 0, 0), 9, 16, 4, 9000, 8999, 32, 0, None),
    ("d256_turbo4k", 256, (32, 4, 0, 0), (32, 3, 0, 0), 6, 8, 2, 700, 655, 64, 64, [64, 1, 0, 9, 33, 64]),
    ("d256_rows_160", 256, (32, 4, 0, 0), (32, 3, 0, 0), 40, 8, 2, 330, 330, 32, 16, None),
    ("d256_gqa8_1bit", 256, (64, 1, 0, 0), (256, 2, 0, 0), 3, 8, 1, 200, 130, 32, 32, None),
    ("d64_pervec_gqa2", 64, (64, 4, 0, 0), (64, 4, 0, 0), 7, 16, 8, 320, 291, 40, 33, [33, 2, 0, 0, 31, 32, 1]),
    ("d64_block32_gqa1", 64, (32, 4, 0, 0), (32, 2, 0, 0), 11, 4, 4, 500, 450, 64, 64, None),
    ("d64_rows_140", 64, (64, 4, 0, 0), (64, 3, 0, 0), 70, 4, 2, 128, 128, 32, 20, None),
    ("beta_nc", 128, (128, 3, 0, 1), (128, 3, 0, 1), 4, 8, 2, 260, 250, 32, 32, None),
    ("pervec_2k3v", 128, (128, 2, 0, 0), (128, 3, 0, 0), 8, 8, 2, 1100, 1100, 128, 100, None),
    # layouts that read the prefix per sequence
    ("qjl_keys", 128, (128, 2, 128, 0), (128, 3, 0, 0), 3, 8, 2, 400, 390, 64, 50, [50, 0, 7]),
    ("qjl_values_gqa2", 128, (128, 2, 128, 0), (128, 2, 128, 0), 2, 4, 2, 200, 200, 32, 32, None),
    ("k8v4", 128, (32, 8, 0, 0), (32, 4, 0, 0), 3, 8, 2, 300, 290, 64, 64, [64, 3, 0]),
    ("k8v4_gqa1_d64", 64, (64, 8, 0, 0), (64, 4, 0, 0), 3, 2, 2, 300, 290, 64, 64, None),
]


def _inputs(tb, d, cK, cV, B, Hq, Hkv, P_cap, cap, seed=1):
    lay = lambda c: tb.make_layout(d, c[0], c[1], c[2], c[3], 1)  # noqa: E731
    S = torch.from_numpy(inputs.qjl_matrix(cK[2], d, 7)).cuda() if cK[2] else None
    Sv = torch.from_numpy(inputs.qjl_matrix(cV[2], d, 8)).cuda() if cV[2] else None
    Kp, Vp = _cache(tb, lay(cK), (1, Hkv, P_cap), seed, S), _cache(tb, lay(cV), (1, Hkv, P_cap), seed + 1, Sv)
    K, V = _cache(tb, lay(cK), (B, Hkv, cap), seed + 2, S), _cache(tb, lay(cV), (B, Hkv, cap), seed + 3, Sv)
    q = torch.from_numpy(inputs.gaussian((B, Hq, d), seed + 4)).cuda()
    return Kp, Vp, K, V, q


@pytest.mark.parametrize("name,d,cK,cV,B,Hq,Hkv,P_cap,prefix,cap,ctx,lens", CASES)
def test_shared_decode_matches_attention_in_64_bits(tqlib, name, d, cK, cV, B, Hq, Hkv, P_cap, prefix, cap, ctx, lens):
    from turboquant_kv_cache_gb300 import binding as tb
    Kp, Vp, K, V, q = _inputs(tb, d, cK, cV, B, Hq, Hkv, P_cap, cap)
    kvl = torch.tensor(lens, dtype=torch.int32, device="cuda") if lens is not None else None
    out = tb.tq_decode_attn_shared(Kp, Vp, K, V, q, prefix_ctx=prefix, ctx=ctx, kv_len=kvl)
    ref = _reference(tb, Kp, Vp, prefix, K, V, [min(n, ctx) for n in (lens or [ctx] * B)], q)
    assert (out.double() - ref).abs().max().item() < ATTN_ATOL, name
    if prefix == 0 and ctx == 0:
        assert not out.any()
    # the same through pages, in another place each
    page = 32 if d == 64 else 64
    Kpp, Ko = _paged(tb, Kp, page, 3), _paged(tb, K, page, 4)
    got = tb.tq_decode_attn_shared(Kpp, _paged(tb, Vp, page, 3, table=Kpp.page_table), Ko,
                                   _paged(tb, V, page, 4, table=Ko.page_table), q, prefix_ctx=prefix, ctx=ctx, kv_len=kvl)
    assert (got.double() - ref).abs().max().item() < ATTN_ATOL, name


@pytest.mark.parametrize("prefix_len", [0, 1, 64, 77, 200, 5000, -3])
def test_prefix_length_on_the_device(tqlib, prefix_len):
    from turboquant_kv_cache_gb300 import binding as tb
    Kp, Vp, K, V, q = _inputs(tb, 128, (32, 3, 0, 0), (32, 3, 0, 0), 4, 8, 2, 256, 32)
    pl = torch.tensor([prefix_len], dtype=torch.int32, device="cuda")
    lens = [32, 0, 5, 17]
    kvl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = tb.tq_decode_attn_shared(Kp, Vp, K, V, q, prefix_ctx=200, prefix_len=pl, ctx=32, kv_len=kvl)
    ref = _reference(tb, Kp, Vp, max(0, min(prefix_len, 200)), K, V, lens, q)
    assert (out.double() - ref).abs().max().item() < ATTN_ATOL
    if prefix_len <= 0:
        assert not out[1].any()   # a sequence without any token


@pytest.mark.parametrize("n_split", [1, 2, 7])
def test_own_split_counts(tqlib, n_split):
    from turboquant_kv_cache_gb300 import binding as tb
    Kp, Vp, K, V, q = _inputs(tb, 128, (32, 3, 0, 0), (32, 3, 0, 0), 4, 8, 2, 512, 700, seed=31)
    out = tb.tq_decode_attn_shared(Kp, Vp, K, V, q, prefix_ctx=500, ctx=666, n_split=n_split)
    ref = _reference(tb, Kp, Vp, 500, K, V, [666] * 4, q)
    assert (out.double() - ref).abs().max().item() < ATTN_ATOL


@pytest.mark.parametrize("d,kbits,vbits,block", [(64, 4, 4, 64), (64, 1, 2, 32), (128, 3, 3, 32), (128, 4, 1, 128),
                                                 (256, 4, 3, 32), (256, 2, 4, 256)])
@pytest.mark.parametrize("ctx", [383, 385, 512, 513, 640, 641, 767, 1408])
def test_slices_of_many_tiles(tqlib, d, kbits, vbits, block, ctx):
    """Own tokens and prefix in one part each, over tile counts from three up,
    and the same output again."""
    from turboquant_kv_cache_gb300 import binding as tb
    Kp, Vp, K, V, q = _inputs(tb, d, (block, kbits, 0, 0), (block, vbits, 0, 0), 40, 8, 2, 1409, 1409, seed=51)
    one = tb.tq_decode_attn_shared(Kp, Vp, K, V, q, prefix_ctx=0, ctx=ctx, n_split=1)
    two = tb.tq_decode_attn_shared(Kp, Vp, K, V, q, prefix_ctx=0, ctx=ctx, n_split=1)
    assert torch.equal(one, two)
    pick = [0, 17, 39]   # sequences checked
    ref = _reference(tb, Kp, Vp, 0, *(tb.PackedKV.of(c.layout, c.codes[pick], c.scales[pick]) for c in (K, V)),
                     [ctx] * 3, q[pick])
    assert (one[pick].double() - ref).abs().max().item() < ATTN_ATOL


def test_oracle_bytes(tqlib):
    """The oracle's own packed bytes and its decoded vectors."""
    from turboquant_kv_cache_gb300 import binding as tb
    B, Hq, Hkv, P, cap, d = 3, 8, 2, 300, 64, 128
    lens = [64, 0, 21]
    Lk, Lv = O.Layout(d, 32, 3), O.Layout(d, 32, 3)
    dev, deq = {}, {}
    for name, lead, L, seed in (("kp", (1, Hkv, P), Lk, 1), ("vp", (1, Hkv, P), Lv, 2), ("k", (B, Hkv, cap), Lk, 3),
                                ("v", (B, Hkv, cap), Lv, 4)):
        c, s, _, _ = O.encode(inputs.gaussian(lead + (d,), seed).reshape(-1, d), L)
        dev[name] = upload_packed(tb, tb.make_layout(d, 32, 3), L, c, s, None, None, lead)
        deq[name] = O.dequantize(c, s, L).reshape(lead + (d,))
    q = inputs.gaussian((B, Hq, d), 5)
    out = tb.tq_decode_attn_shared(dev["kp"], dev["vp"], dev["k"], dev["v"], torch.from_numpy(q).cuda(), prefix_ctx=P,
                                   ctx=cap, kv_len=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    for b in range(B):
        k = np.concatenate([deq["kp"], deq["k"][b:b + 1, :, :lens[b]]], 2)
        v = np.concatenate([deq["vp"], deq["v"][b:b + 1, :, :lens[b]]], 2)
        ref = O.decode_attention(q[b:b + 1], k, v)
        assert np.abs(to_np(out[b:b + 1]).astype(np.float64) - ref).max() < ATTN_ATOL


def test_scale_and_long_scores(tqlib):
    """A softmax scale of the caller's, with scores far apart: the parts'
    maxima differ by hundreds, and their merge stays finite."""
    from turboquant_kv_cache_gb300 import binding as tb
    Kp, Vp, K, V, q = _inputs(tb, 128, (32, 4, 0, 0), (32, 3, 0, 0), 4, 8, 2, 300, 64, seed=61)
    out = tb.tq_decode_attn_shared(Kp, Vp, K, V, q, prefix_ctx=300, ctx=64, softmax_scale=4.0)
    ref = _reference(tb, Kp, Vp, 300, K, V, [64] * 4, q, 4.0)
    assert torch.isfinite(out).all()
    # scores reach 4 * 128 * ... = hundreds, so a score's fp16 operand
    # roundings (2 * 2^-11 relative, of sums of |q k| up to 4 * 100) move a
    # weight by up to e^0.4: only the rows' winner is certain
    best = _reference(tb, Kp, Vp, 300, K, V, [64] * 4, q, 400.0)
    far = (out.double() - ref).abs().amax(-1)
    sure = (ref - best).abs().amax(-1) < 1e-6
    assert (far[sure] < 2e-2).all()


def test_views_into_one_table(tqlib):
    """Prefix and own pages in one pool and one table: the own view is the
    table's columns behind the prefix's pages."""
    from turboquant_kv_cache_gb300 import binding as tb
    B, Hq, Hkv, d, page, pre, own = 4, 8, 2, 128, 32, 5, 2
    Kp, Vp, K, V, q = _inputs(tb, d, (32, 3, 0, 0), (32, 3, 0, 0), B, Hq, Hkv, pre * page, own * page, seed=71)
    n = pre + B * own + 3
    perm = np.random.default_rng(9).permutation(n).astype(np.int32)
    table = np.empty((B, pre + own), np.int32)
    table[:, :pre] = perm[:pre]
    table[:, pre:] = perm[pre:pre + B * own].reshape(B, own)
    dt = torch.from_numpy(table).cuda()
    whole = {}
    for name, Cp, C in (("k", Kp, K), ("v", Vp, V)):
        P = tb.PackedKV(C.layout, (n, Hkv, page), page_table=dt)
        for arr in ("codes", "scales"):
            dst = getattr(P, arr)
            dst.zero_()
            for j in range(pre):
                dst[int(table[0, j])] = getattr(Cp, arr)[0, :, j * page:(j + 1) * page]
            for b in range(B):
                for j in range(own):
                    dst[int(table[b, pre + j])] = getattr(C, arr)[b, :, j * page:(j + 1) * page]
        whole[name] = P
    part = lambda P, t: tb.PackedKV.of(P.layout, P.codes, P.scales, page_table=t)  # noqa: E731
    args = [part(whole["k"], dt[:1, :pre]), part(whole["v"], dt[:1, :pre]), part(whole["k"], dt[:, pre:]),
            part(whole["v"], dt[:, pre:])]
    kvl = torch.tensor([64, 1, 0, 40], dtype=torch.int32, device="cuda")
    out = tb.tq_decode_attn_shared(*args, q, prefix_ctx=pre * page, ctx=own * page, kv_len=kvl)
    ref = _reference(tb, Kp, Vp, pre * page, K, V, kvl.tolist(), q)
    assert (out.double() - ref).abs().max().item() < ATTN_ATOL
    # and the decode over the whole table says the same
    dec = tb.tq_decode_attn(whole["k"], whole["v"], q, ctx=(pre + own) * page, kv_len=kvl + pre * page)
    assert (dec.double() - ref).abs().max().item() < ATTN_ATOL


def test_captured_replays_and_two_streams(tqlib):
    """A captured call replayed with other inputs and lengths, and calls on
    two streams with a workspace each, give what eager calls give."""
    from turboquant_kv_cache_gb300 import binding as tb
    Kp, Vp, K, V, q = _inputs(tb, 128, (32, 3, 0, 0), (32, 3, 0, 0), 6, 8, 2, 512, 64, seed=81)
    pl = torch.tensor([512], dtype=torch.int32, device="cuda")
    kvl = torch.full((6,), 64, dtype=torch.int32, device="cuda")
    ws = torch.empty(tb.tq_decode_shared_workspace_bytes(6, 8, 2, 128, 512, 64), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    call = lambda o, w, s=None: tb.tq_decode_attn_shared(Kp, Vp, K, V, q, prefix_ctx=512, prefix_len=pl, ctx=64,  # noqa: E731
                                                         kv_len=kvl, workspace=w, out=o, stream=s)
    call(out, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out, ws)
    for n, m in ((512, 64), (100, 3), (0, 64), (64, 0)):
        pl.fill_(n)
        kvl.fill_(m)
        q.copy_(torch.from_numpy(inputs.gaussian((6, 8, 128), 90 + n)).cuda())
        out.fill_(float("nan"))
        g.replay()
        eager = call(torch.empty_like(q), torch.empty_like(ws))
        torch.cuda.synchronize()
        assert torch.equal(out, eager), (n, m)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    o1, o2, w2 = torch.empty_like(q), torch.empty_like(q), torch.empty_like(ws)
    for _ in range(5):
        s1.wait_stream(torch.cuda.current_stream())
        s2.wait_stream(torch.cuda.current_stream())
        call(o1, ws, s1)
        call(o2, w2, s2)
    torch.cuda.synchronize()
    assert torch.equal(o1, eager) and torch.equal(o2, eager)


def test_binding_refusals(tqlib):
    from turboquant_kv_cache_gb300 import binding as tb
    Kp, Vp, K, V, q = _inputs(tb, 128, (32, 3, 0, 0), (32, 3, 0, 0), 2, 8, 2, 64, 64)
    with pytest.raises(ValueError):
        tb.tq_decode_attn_shared(Kp, Vp, K, V, q.float())
    with pytest.raises(ValueError):
        tb.tq_decode_attn_shared(Kp, Vp, K, V, q, kv_len=torch.ones(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        tb.tq_decode_attn_shared(Kp, Vp, K, V, q, prefix_len=torch.ones(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        tb.tq_decode_attn_shared(Kp, Vp, K, V, q, out=torch.empty(2, 8, 64, dtype=torch.float16, device="cuda"))
    with pytest.raises(tb.TQError):
        tb.tq_decode_attn_shared(Kp, Vp, K, V, q, prefix_ctx=65)


@pytest.mark.parametrize("B,Hq,Hkv,d,short", [(7, 16, 8, 64, (300, 200)), (2, 8, 2, 128, (1, 9)), (4, 4, 1, 256, (1500, 0))])
def test_workspace_of_longer_lengths(tqlib, B, Hq, Hkv, d, short):
    """A workspace for the longest lengths serves shorter ones, with the same results."""
    from turboquant_kv_cache_gb300 import binding as tb
    L = (32, 3, 0, 0)
    Kp, Vp, K, V, q = _inputs(tb, d, L, L, B, Hq, Hkv, 2048, 512)
    ws = torch.empty(tb.tq_decode_shared_workspace_bytes(B, Hq, Hkv, d, 2048, 512), dtype=torch.uint8, device="cuda")
    for P, S in [(2048, 512), short, (0, 512), (2048, 0)]:
        got = tb.tq_decode_attn_shared(Kp, Vp, K, V, q, prefix_ctx=P, ctx=S, workspace=ws)
        assert torch.equal(got, tb.tq_decode_attn_shared(Kp, Vp, K, V, q, prefix_ctx=P, ctx=S))
        ref = _reference(tb, Kp, Vp, P, K, V, [S] * B, q)
        assert (got.double() - ref).abs().max().item() < ATTN_ATOL


def test_reports_timeout_and_stays_exact(tqlib):
    """A wait limit far below any real wait (1 ns): TQ_ERR_TIMEOUT in the
    device status, the output that of an ordinary launch."""
    from turboquant_kv_cache_gb300 import binding as tb
    L = (32, 3, 0, 0)
    Kp, Vp, K, V, q = _inputs(tb, 128, L, L, 8, 32, 8, 4096, 256)
    run = lambda: tb.tq_decode_attn_shared(Kp, Vp, K, V, q, prefix_ctx=4000, ctx=250)  # noqa: E731
    torch.cuda.synchronize()
    tb.tq_set_wait_limit_ns(0)
    tb.tq_device_status(clear=True)
    try:
        ref = run()
        assert tb.tq_device_status(clear=True) == 0
        tb.tq_set_wait_limit_ns(1)
        got = run()
        assert tb.tq_device_status(clear=True) == -6
        assert torch.equal(got, ref)
    finally:
        tb.tq_set_wait_limit_ns(0)
        tb.tq_device_status(clear=True)
    assert torch.equal(run(), ref)
    assert tb.tq_device_status() == 0


@pytest.mark.parametrize("paged", [False, True])
def test_offsets_past_32_bits(tqlib, paged):
    """A prefix and own tokens that lie more than 2^32 bytes into their
    arrays give what the same records give in small arrays."""
    from turboquant_kv_cache_gb300 import binding as tb
    d, B, Hq, Hkv, P, S = 256, 2, 8, 4, 700, 90
    Kp, Vp, K, V, q = _inputs(tb, d, (32, 4, 0, 0), (32, 3, 0, 0), B, Hq, Hkv, P, S)
    want = tb.tq_decode_attn_shared(Kp, Vp, K, V, q)

    def far(c, table):
        n = c.lead_shape[0]
        if paged:   # pages of 32 tokens at the end of a pool of 2^33 bytes of codes (K) and less
            page, pps = 32, -(-c.lead_shape[2] // 32)
            pool = (1 << 33) // (Hkv * page * 128) + n * pps
            lead = (pool, Hkv, page)
        else:       # heads 2^31 bytes apart and more
            lead = (n, Hkv, (1 << 31) // 96 + 1)
        codes = torch.empty(lead + c.codes.shape[3:], dtype=torch.uint8, device="cuda")
        scales = torch.empty(lead + c.scales.shape[3:], dtype=torch.float16, device="cuda")
        for src, dst in ((c.codes, codes), (c.scales, scales)):
            for b in range(n):
                if not paged:
                    dst[b, :, :c.lead_shape[2]] = src[b]
                    continue
                for j in range(pps):
                    part = src[b, :, 32 * j:32 * j + 32]
                    dst[pool - n * pps + b * pps + j, :, :part.shape[1]] = part
        if paged and table is None:
            table = (torch.arange(n * pps, dtype=torch.int32, device="cuda") + (pool - n * pps)).view(n, pps)
        return tb.PackedKV.of(c.layout, codes, scales, page_table=table)

    Kp2 = far(Kp, None)
    Vp2 = far(Vp, Kp2.page_table)
    assert torch.equal(tb.tq_decode_attn_shared(Kp2, Vp2, K, V, q, prefix_ctx=P), want)
    del Kp2, Vp2
    K2 = far(K, None)
    V2 = far(V, K2.page_table)
    assert torch.equal(tb.tq_decode_attn_shared(Kp, Vp, K2, V2, q, ctx=S), want)


def test_one_own_cache_alone_is_refused(tqlib):
    """K without V (or V without K) is no batch without own tokens."""
    from turboquant_kv_cache_gb300 import binding as tb
    Kp, Vp, K, V, q = _inputs(tb, 128, (32, 3, 0, 0), (32, 3, 0, 0), 2, 8, 2, 64, 64)
    for k, v in ((K, None), (None, V)):
        for kw in (dict(), dict(ctx=0), dict(ctx=64)):
            with pytest.raises(ValueError):
                tb.tq_decode_attn_shared(Kp, Vp, k, v, q, **kw)
    ref = _reference(tb, Kp, Vp, 64, None, None, None, q)
    assert (tb.tq_decode_attn_shared(Kp, Vp, None, None, q).double() - ref).abs().max().item() < ATTN_ATOL
