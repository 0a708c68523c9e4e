"""tq_qkv_norm_rope against the same formulas in 64 bits.

The kernel computes in fp32 and rounds once to fp16.  Its error is then half
an fp16 step, 2^-11 of the value (2^-25 below the normal range), and the fp32
steps before it: a sum of at most 256 squares by a thread's eight and a
butterfly of five (13 roundings), a mean, a reciprocal square root (2 steps)
and two products, so a factor off by at most 20 * 2^-24; the rotation's two
products and sum add three roundings of |a| + |b|.  24 * 2^-24 of |a| + |b|
bounds the fp32 part, where a and b are a value and its pair's other one."""
import numpy as np
import pytest
import torch

from turboquant_kv_cache_gb300 import inputs

pytestmark = pytest.mark.gpu

HALF_STEP, F32 = 2.0 ** -11, 24 * 2.0 ** -24


def _table(n_pos, rot):
    ang = np.arange(n_pos)[:, None] * 1e4 ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def _reference(x, Hq, Hkv, d, wq, wk, eps, table, inter, pos):
    """(values, |a| + |b|) of the rows x [B, T, H, d] in 64 bits."""
    x = x.astype(np.float64)
    B, T = x.shape[:2]
    y = x.copy()
    for lo, hi, w in ((0, Hq, wq), (Hq, Hq + Hkv, wk)):
        if w is not None:
            z = x[:, :, lo:hi]
            y[:, :, lo:hi] = z / np.sqrt((z ** 2).mean(-1, keepdims=True) + eps) * w.astype(np.float64)
    size = np.abs(y)
    if table is not None:
        rot = table.shape[1]
        n = rot // 2
        i = np.arange(n)
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + n)
        p = np.clip(pos[:, None] + np.arange(T), 0, table.shape[0] - 1)
        c, s = (t[:, :, None] for t in np.split(table.astype(np.float64)[p], 2, axis=-1))
        u, v = y[:, :, :Hq + Hkv, a].copy(), y[:, :, :Hq + Hkv, b].copy()
        y[:, :, :Hq + Hkv, a], y[:, :, :Hq + Hkv, b] = u * c - v * s, v * c + u * s
        size[:, :, :Hq + Hkv, a] = size[:, :, :Hq + Hkv, b] = np.abs(u) + np.abs(v)
    return y, size


def _near(got, ref, size):
    err = np.abs(got.double().cpu().numpy() - ref)
    tol = HALF_STEP * np.abs(ref) + F32 * size + 2.0 ** -25
    assert (err <= tol).all(), float((err / tol).max())


CASES = [
    # B, T, Hq, Hkv, d, fp32, rot, interleaved, norm of q, norm of k, cap extra
    (8, 1, 32, 8, 128, False, 128, False, True, True, 3),
    (1, 1, 1, 1, 64, False, 64, False, True, True, 0),
    (3, 5, 7, 1, 256, True, 256, False, True, True, 0),
    (2, 7, 16, 4, 256, False, 64, True, True, True, 1),
    (2, 33, 8, 8, 64, True, 32, True, True, False, 0),
    (1, 130, 4, 2, 128, False, 96, False, False, True, 0),
    (2, 9, 5, 3, 128, False, 48, False, True, True, 2),
    (2, 9, 5, 3, 128, True, 16, True, False, False, 2),
    (1, 3, 24, 8, 64, False, 0, False, True, True, 0),
    (1, 2, 3, 1, 256, False, 0, False, False, False, 5),
    (5, 701, 8, 4, 64, False, 64, False, False, False, 0),
]


@pytest.mark.parametrize("B,T,Hq,Hkv,d,f32,rot,inter,nq,nk,extra", CASES)
def test_rows_match_64_bits(tqlib, B, T, Hq, Hkv, d, f32, rot, inter, nq, nk, extra):
    from turboquant_kv_cache_gb300 import binding as tb
    H = Hq + 2 * Hkv
    x = inputs.gaussian((B, T, H * d), 1, np.float32) * np.exp(inputs.gaussian((H * d,), 2, np.float32))
    x = x if f32 else x.astype(np.float16)
    w = 1 + 0.2 * inputs.gaussian((2, d), 3, np.float32)
    wq, wk = (w[0] if nq else None), (w[1] if nk else None)
    table = _table(500 + T, rot) if rot else None
    rng = np.random.default_rng(4)
    pos = rng.integers(0, 500, B).astype(np.int32)
    slot = rng.integers(0, extra + 1, B).astype(np.int32)
    cu = lambda a: torch.from_numpy(a).cuda() if a is not None else None  # noqa: E731
    cap = T + extra
    k = torch.full((B, Hkv, cap, d), 9.0, dtype=torch.float16, device="cuda")
    v = torch.full((B, Hkv, cap, d), 9.0, dtype=torch.float16, device="cuda")
    q, k, v = tb.tq_qkv_norm_rope(cu(x), Hq, Hkv, d, cu(wq), cu(wk), 1e-5, cu(table), inter, cu(pos), slot=cu(slot),
                                  k_out=k, v_out=v)
    ref, size = _reference(x.reshape(B, T, H, d), Hq, Hkv, d, wq, wk, 1e-5, table, inter, pos)
    order = lambda a: a.transpose(0, 2, 1, 3)  # noqa: E731
    _near(q, order(ref[:, :, :Hq]), order(size[:, :, :Hq]))
    for b in range(B):
        at = slice(slot[b], slot[b] + T)
        _near(k[b, :, at], order(ref[b:b + 1, :, Hq:Hq + Hkv])[0], order(size[b:b + 1, :, Hq:Hq + Hkv])[0])
        _near(v[b, :, at], order(ref[b:b + 1, :, Hq + Hkv:])[0], order(size[b:b + 1, :, Hq + Hkv:])[0])
        for o in (k, v):   # the other slots are as they were
            rest = torch.ones(cap, dtype=torch.bool)
            rest[at] = False
            assert (o[b, :, rest.cuda()] == 9.0).all()


def test_padded_batch_and_positions_outside_the_table(tqlib):
    """Tokens behind new_len, tokens whose position has no table row and slots
    outside the arrays leave everything as it was; padding may hold NaN."""
    from turboquant_kv_cache_gb300 import binding as tb
    B, T, Hq, Hkv, d = 5, 6, 3, 2, 128
    x = inputs.gaussian((B, T, (Hq + 2 * Hkv) * d), 5)
    lens = np.array([6, 0, 3, 9, -2], np.int32)
    pos = np.array([0, 0, 7, -2, 3], np.int32)      # table of 9 rows
    slot = np.array([-1, 0, 4, 2, 0], np.int32)     # cap 6
    table = _table(9, d)
    x[2, 3:] = np.nan
    cu = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    mk = lambda *s: torch.full(s, 9.0, dtype=torch.float16, device="cuda")  # noqa: E731
    q, k, v = tb.tq_qkv_norm_rope(cu(x), Hq, Hkv, d, None, None, rope=cu(table), pos=cu(pos), new_len=cu(lens),
                                  slot=cu(slot), q_out=mk(B, Hq, T, d), k_out=mk(B, Hkv, T, d), v_out=mk(B, Hkv, T, d))
    ref, size = _reference(x.reshape(B, T, -1, d), Hq, Hkv, d, None, None, 1e-6, table, False, pos)
    for b in range(B):
        done = set()
        for j in range(T):
            live = j < lens[b] and 0 <= pos[b] + j < 9
            if live:
                _near(q[b, :, j], ref[b, j, :Hq], size[b, j, :Hq])
            else:
                assert (q[b, :, j] == 9.0).all()
            s = slot[b] + j
            if live and 0 <= s < T:
                done.add(s)
                _near(k[b, :, s], ref[b, j, Hq:Hq + Hkv], size[b, j, Hq:Hq + Hkv])
                _near(v[b, :, s], ref[b, j, Hq + Hkv:], size[b, j, Hq + Hkv:])
        for s in set(range(T)) - done:
            assert (k[b, :, s] == 9.0).all() and (v[b, :, s] == 9.0).all()


def test_strided_rows_and_special_values(tqlib):
    """Rows cut out of a wider projection; zero rows give zeros under a norm,
    infinities and NaN stay in their own head."""
    from turboquant_kv_cache_gb300 import binding as tb
    B, T, Hq, Hkv, d = 2, 3, 2, 1, 64
    width = (Hq + 2 * Hkv) * d
    wide = torch.from_numpy(inputs.gaussian((B, T, width + 128), 6)).cuda()
    wide[..., 64:64 + width][0, 0, :d] = 0
    wide[..., 64:64 + width][1, 2, d] = float("inf")
    wide[..., 64:64 + width][1, 1, 0] = float("nan")
    x = wide[..., 64:64 + width]
    w = torch.ones(d, device="cuda")
    table = torch.from_numpy(_table(8, d)).cuda()
    a = tb.tq_qkv_norm_rope(x, Hq, Hkv, d, w, w, rope=table)
    b = tb.tq_qkv_norm_rope(x.contiguous(), Hq, Hkv, d, w, w, rope=table)
    for s, t in zip(a, b):
        assert torch.equal(s.view(torch.int16), t.view(torch.int16))
    q, k, v = a
    assert (q[0, 0, 0] == 0).all()
    assert q[1, 1, 2].isnan().any() and q[1, 0, 1].isnan().any()
    q[1, 1, 2] = q[1, 0, 1] = 0
    assert torch.isfinite(q).all() and torch.isfinite(k).all() and torch.isfinite(v).all()


def test_far_offsets_pass_32_bits(tqlib):
    """Outputs whose element offsets pass 2^31."""
    from turboquant_kv_cache_gb300 import binding as tb
    B, T, Hq, Hkv, d, cap = 2, 1, 1, 1, 256, 8_600_000
    x = torch.from_numpy(inputs.gaussian((B, T, 3 * d), 8)).cuda()
    k = torch.zeros(B, Hkv, cap, d, dtype=torch.float16, device="cuda")
    v = torch.zeros_like(k)
    slot = torch.tensor([0, cap - 1], dtype=torch.int32, device="cuda")
    tb.tq_qkv_norm_rope(x, Hq, Hkv, d, slot=slot, k_out=k, v_out=v)
    assert torch.equal(k[1, 0, cap - 1], x[1, 0, d:2 * d]) and torch.equal(v[1, 0, cap - 1], x[1, 0, 2 * d:])
    assert not k[1, 0, :cap - 1].any() and not v[0, 0, 1:].any()


def test_rows_feed_append_and_window(tqlib):
    """What it writes is what tq_append_kv and tq_decode_attn_window take."""
    from turboquant_kv_cache_gb300 import binding as tb
    B, T, Hq, Hkv, d = 2, 40, 8, 2, 128
    x = torch.from_numpy(inputs.gaussian((B, T, (Hq + 2 * Hkv) * d), 9)).cuda()
    w = torch.ones(d, device="cuda")
    q, k, v = tb.tq_qkv_norm_rope(x, Hq, Hkv, d, w, w, rope=torch.from_numpy(_table(T, d)).cuda())
    L = tb.make_layout(d, 32, 4)
    K, V = tb.PackedKV(L, (B, Hkv, 64)), tb.PackedKV(L, (B, Hkv, 64))
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    tb.tq_append_kv(K, k, zero)
    tb.tq_append_kv(V, v, zero)
    one = q[:, :, T - 1].contiguous()
    packed = tb.tq_decode_attn(K, V, one, ctx=T)
    window = tb.tq_decode_attn_window(K, V, one, k, v, ctx=64, kv_len=zero)
    s = torch.einsum("bhd,bhtd->bht", one.double(), k.double().repeat_interleave(Hq // Hkv, 1)) / d ** 0.5
    ref = torch.einsum("bht,bhtd->bhd", s.softmax(-1), v.double().repeat_interleave(Hq // Hkv, 1))
    assert (window.double() - ref).abs().max().item() < 2e-3
    # 4-bit codes keep a vector to about 10% of its norm; the attention of 40
    # such values with unit entries stays within their mean error
    assert (packed.double() - ref).abs().mean().item() < 0.1
    g = torch.cuda.CUDAGraph()
    out = [torch.zeros_like(t) for t in (q, k, v)]
    args = dict(rope=torch.from_numpy(_table(T, d)).cuda(), q_out=out[0], k_out=out[1], v_out=out[2])
    tb.tq_qkv_norm_rope(x, Hq, Hkv, d, w, w, **args)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        tb.tq_qkv_norm_rope(x, Hq, Hkv, d, w, w, **args)
    for o in out:
        o.zero_()
    g.replay()
    for o, t in zip(out, (q, k, v)):
        assert torch.equal(o, t)


def test_binding_refusals(tqlib):
    from turboquant_kv_cache_gb300 import binding as tb
    x = torch.zeros(2, 3, 5 * 64, dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError):
        tb.tq_qkv_norm_rope(x, 4, 1, 64)
    with pytest.raises(ValueError):
        tb.tq_qkv_norm_rope(x, 3, 1, 64, pos=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        tb.tq_qkv_norm_rope(x, 3, 1, 64, q_weight=torch.ones(64, dtype=torch.float16, device="cuda"))
    with pytest.raises(TypeError):
        tb.tq_qkv_norm_rope(x.bfloat16(), 3, 1, 64)
    with pytest.raises(tb.TQError):
        tb.tq_qkv_norm_rope(x, 3, 1, 64, rope=torch.zeros(8, 24, device="cuda"))


@pytest.mark.parametrize("kw", [dict(), dict(new_len=[7, 2]), dict(pos=[30, 5]), dict(slot=[3, -2]), dict(rows=5),
                                dict(cap=16), dict(cap=4)])
def test_new_outputs_are_zero_where_no_token_goes(tqlib, kw):
    """Outputs that the call makes, over memory that held something else: a
    rotation table of fewer rows than there are tokens leaves tokens out with
    no other argument, and new values beside given keys have the keys' slots."""
    from turboquant_kv_cache_gb300 import binding as tb
    B, T, Hq, Hkv, d = 2, 9, 3, 2, 64
    x = torch.from_numpy(inputs.gaussian((B, T, (Hq + 2 * Hkv) * d), 31)).cuda()
    rope = torch.from_numpy(_table(kw.get("rows", 32), d)).cuda()
    args = {n: torch.tensor(kw[n], dtype=torch.int32, device="cuda") for n in ("new_len", "pos", "slot") if n in kw}
    cap = kw.get("cap")
    z = lambda *s: torch.zeros(s, dtype=torch.float16, device="cuda")  # noqa: E731
    want = tb.tq_qkv_norm_rope(x, Hq, Hkv, d, rope=rope, q_out=z(B, Hq, T, d), k_out=z(B, Hkv, cap or T, d),
                               v_out=z(B, Hkv, cap or T, d), **args)
    k_out = z(B, Hkv, cap, d) if cap else None
    for h in (Hq, Hkv, Hkv):     # what the allocator hands out next
        for n in (T, cap or T):
            torch.full((B, h, n, d), 9.0, dtype=torch.float16, device="cuda")
    got = tb.tq_qkv_norm_rope(x, Hq, Hkv, d, rope=rope, k_out=k_out, **args)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


# Thread groups that take several rows of a token: 4 rows (12 heads; 7 and 11
# with one group's last head missing), 3 (9 heads; 5 with one missing), 2 (10
# heads; 13 with one missing), with the borders between query, key and value
# heads inside a group.  There are enough tokens for 2432 blocks of one row.
GROUPS = [
    # rows a group, B, T, Hq, Hkv, d
    (4, 5, 401, 6, 3, 128), (4, 3, 1201, 3, 2, 128), (4, 3, 301, 5, 3, 256), (4, 4, 900, 6, 3, 64),
    (3, 5, 451, 5, 2, 128), (3, 4, 601, 3, 1, 256), (2, 5, 401, 4, 3, 128), (2, 3, 301, 7, 3, 256),
]


@pytest.mark.parametrize("rows,B,T,Hq,Hkv,d", GROUPS)
@pytest.mark.parametrize("f32,rot,inter,nq,nk", [(False, 1.0, False, True, True), (True, 0.5, True, True, True),
                                                 (False, 0.75, True, True, False), (True, 1.0, False, False, True),
                                                 (False, 0.0, False, True, True)])
def test_groups_of_several_rows(tqlib, rows, B, T, Hq, Hkv, d, f32, rot, inter, nq, nk):
    H = Hq + 2 * Hkv
    idle = {r: -H % r for r in (4, 3, 2)}
    assert -(-B * T // (64 // (d // 16))) * H > 152 * 16 and min(idle, key=idle.get) == rows   # the library's rule
    test_rows_match_64_bits(tqlib, B, T, Hq, Hkv, d, f32, int(rot * d) // 16 * 16, inter, nq, nk, 2)


@pytest.mark.parametrize("Hq,Hkv,d,f32", [(6, 3, 128, False), (5, 2, 256, True), (7, 3, 64, False)])
def test_groups_of_several_rows_in_a_padded_batch(tqlib, Hq, Hkv, d, f32):
    """Ragged lengths over many tokens: the tokens there are as without
    lengths, the rest is left alone."""
    from turboquant_kv_cache_gb300 import binding as tb
    B, T = 6, 900
    x = torch.from_numpy(inputs.gaussian((B, T, (Hq + 2 * Hkv) * d), 41, np.float32 if f32 else np.float16)).cuda()
    w = torch.from_numpy(1 + 0.2 * inputs.gaussian((2, d), 42, np.float32)).cuda()
    rope = torch.from_numpy(_table(T, d)).cuda()
    full = tb.tq_qkv_norm_rope(x, Hq, Hkv, d, w[0], w[1], rope=rope)
    lens = [900, 0, 1, 899, 450, 7]
    outs = [torch.full_like(t, 9.0) for t in full]
    pad = x.clone()
    for b, n in enumerate(lens):
        pad[b, n:] = float("nan")
    tb.tq_qkv_norm_rope(pad, Hq, Hkv, d, w[0], w[1], rope=rope, new_len=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                        q_out=outs[0], k_out=outs[1], v_out=outs[2])
    for o, t in zip(outs, full):
        for b, n in enumerate(lens):
            assert torch.equal(o[b, :, :n], t[b, :, :n]) and (o[b, :, n:] == 9.0).all()
