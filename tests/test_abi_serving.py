"""Argument checks of the shared-prefix decode, the query/key norm with
rotary position and the page-table calls: every refusal happens on the host,
so none of this needs a GPU."""
import ctypes

import pytest

from turboquant_kv_cache_gb300 import binding as tb

P16 = ctypes.c_void_p(16)
P8 = ctypes.c_void_p(8)
ARG, UNSUP, ALIGN, WORKSPACE = -1, -2, -3, -4


def _view(L, table=None, page=0, pps=0, ptr=16):
    return tb.tq_kv_view(ptr, 16, None, None, None, L, table, page, pps)


def _shared(lib, Kp=None, Vp=None, K=None, V=None, P_cap=128, prefix=100, B=2, Hq=8, Hkv=2, S_cap=64, ctx=50, q=P16,
            out=P16, ws=P16, nbytes=1 << 24, n_split=0):
    L = tb.make_layout(128, 32, 3)
    views = [v if v is not None else _view(L) for v in (Kp, Vp, K, V)]
    refs = [ctypes.byref(v) if v != "null" else None for v in views]
    return lib.tq_decode_attn_shared(refs[0], refs[1], P_cap, None, prefix, refs[2], refs[3], q, B, Hq, Hkv, S_cap, None,
                                     ctx, 0.0, out, ws, nbytes, n_split, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), ARG), (dict(out=None), ARG), (dict(Kp="null"), ARG), (dict(Vp="null"), ARG), (dict(K="null"), ARG),
    (dict(prefix=129), ARG), (dict(prefix=-1), ARG), (dict(ctx=65), ARG), (dict(ctx=-1), ARG), (dict(B=0), ARG),
    (dict(Hq=7), ARG), (dict(n_split=-1), ARG), (dict(Hq=6), UNSUP), (dict(Hq=32), UNSUP), (dict(B=40000), UNSUP),
    (dict(q=P8), ALIGN), (dict(out=P8), ALIGN), (dict(ws=P8), ALIGN), (dict(ws=None), WORKSPACE),
    (dict(nbytes=64), WORKSPACE),
    (dict(K=_view(tb.make_layout(128, 32, 4))), ARG),                       # another layout than the prefix's
    (dict(V=_view(tb.make_layout(128, 32, 3, sign_seed=2))), ARG),
    (dict(Vp=_view(tb.make_layout(64, 32, 3))), UNSUP),
    (dict(Vp=_view(tb.make_layout(128, 32, 8))), UNSUP),
    (dict(Kp=_view(tb.make_layout(128, 32, 3), table=16, page=32, pps=2)), ARG),   # 64 slots of pages for 128
    (dict(Kp=_view(tb.make_layout(128, 32, 3), table=16, page=48, pps=4)), ARG),   # page size no multiple of 32
    (dict(K=_view(tb.make_layout(128, 32, 3), table=16, page=64, pps=2)), ARG),    # K paged, V not
    (dict(Kp=_view(tb.make_layout(128, 32, 3), ptr=8)), ALIGN),
    (dict(V=_view(tb.make_layout(128, 32, 3), ptr=8)), ALIGN),
    (dict(Kp=_view(tb.make_layout(128, 32, 3), ptr=None)), ARG),
])
def test_shared_decode_refusals(tqlib, kw, status):
    assert _shared(tqlib, **kw) == status


def test_shared_workspace_query(tqlib):
    nb = ctypes.c_size_t()
    q = lambda *a: tqlib.tq_decode_shared_workspace_bytes(*a, ctypes.byref(nb))  # noqa: E731
    assert q(8, 32, 8, 128, 32768, 256, 0) == 0
    both = nb.value
    assert q(8, 32, 8, 128, 0, 256, 0) == 0 and nb.value < both
    assert q(8, 32, 8, 128, -1, 256, 0) == ARG
    assert q(8, 32, 8, 96, 1, 1, 0) == UNSUP
    assert q(8, 32, 7, 128, 1, 1, 0) == ARG
    assert tqlib.tq_decode_shared_workspace_bytes(8, 32, 8, 128, 1, 1, 0, None) == ARG


@pytest.mark.parametrize("B,Hq,Hkv,d", [(1, 1, 1, 64), (7, 16, 8, 64), (4, 32, 8, 128), (8, 16, 4, 256), (64, 8, 1, 128)])
def test_shared_workspace_serves_shorter_lengths(tqlib, B, Hq, Hkv, d):
    def need(P, S):
        nb = ctypes.c_size_t()
        assert tqlib.tq_decode_shared_workspace_bytes(B, Hq, Hkv, d, P, S, 0, ctypes.byref(nb)) == 0
        return nb.value

    lengths = [0, 1, 128, 129, 500, 2000, 9000, 40000, 200000]
    for S in lengths:
        for a, b in zip(lengths, lengths[1:]):
            assert need(a, S) <= need(b, S)
            assert need(S, a) <= need(S, b)


def _rows(lib, x=P16, dt=0, B=1, T=2, Hq=8, Hkv=2, d=128, stride=None, wq=P16, wk=P16, eps=1e-6, rope=P16, n_pos=10,
          rot=128, inter=0, q=P16, k=P16, v=P16, cap=2):
    stride = (Hq + 2 * Hkv) * d if stride is None else stride
    return lib.tq_qkv_norm_rope(x, dt, B, T, Hq, Hkv, d, stride, wq, wk, eps, rope, n_pos, rot, inter, None, None, q, k,
                                v, cap, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), ARG), (dict(T=-1), ARG), (dict(Hq=0), ARG), (dict(Hkv=0), ARG), (dict(cap=-1), ARG), (dict(d=96), UNSUP),
    (dict(dt=2), ARG), (dict(inter=2), ARG), (dict(rot=144), ARG), (dict(rot=-16), ARG), (dict(rot=24), UNSUP),
    (dict(rope=None), ARG), (dict(n_pos=0), ARG), (dict(eps=0.0), ARG), (dict(eps=float("nan")), ARG),
    (dict(stride=128), ARG), (dict(x=None), ARG), (dict(q=None), ARG), (dict(k=None), ARG), (dict(v=None), ARG),
    (dict(x=P8), ALIGN), (dict(q=P8), ALIGN), (dict(k=P8), ALIGN), (dict(v=P8), ALIGN), (dict(wq=P8), ALIGN),
    (dict(wk=P8), ALIGN), (dict(rope=P8), ALIGN), (dict(stride=12 * 128 + 4), ALIGN), (dict(B=1 << 16, T=1 << 16), UNSUP),
])
def test_norm_rope_refusals(tqlib, kw, status):
    assert _rows(tqlib, **kw) == status


def test_norm_rope_without_tokens_is_a_no_op(tqlib):
    assert _rows(tqlib, B=0, x=None, q=None, k=None, v=None) == 0
    assert _rows(tqlib, T=0, x=None, q=None, k=None, v=None) == 0


def _pool(**kw):
    f = dict(page_table=16, n_pages=16, ref=16, n_seqs=4, pages_per_seq=8, num_pages=32, page_size=64)
    f.update(kw)
    return tb.tq_page_pool(*f.values())


BAD_POOLS = [(dict(page_table=None), ARG), (dict(n_pages=None), ARG), (dict(ref=None), ARG), (dict(n_seqs=0), ARG),
             (dict(pages_per_seq=0), ARG), (dict(num_pages=0), ARG), (dict(page_size=0), ARG), (dict(page_size=48), ARG),
             (dict(pages_per_seq=(1 << 20) + 1), UNSUP), (dict(num_pages=(1 << 28) + 1), UNSUP)]


@pytest.mark.parametrize("kw,status", BAD_POOLS)
def test_bad_pools_are_refused(tqlib, kw, status):
    p = ctypes.byref(_pool(**kw))
    assert tqlib.tq_pages_free(p, P16, None, 1, None) == status
    assert tqlib.tq_pages_fork(p, None, 0, 0, P16, P16, P16, P16, 1, None, P16, 1 << 30, None) == status
    assert tqlib.tq_pages_compact(p, None, 0, 0, None, P16, 1 << 30, None) == status


def test_page_call_refusals(tqlib):
    p = ctypes.byref(_pool())
    assert tqlib.tq_pages_free(None, P16, None, 1, None) == ARG
    assert tqlib.tq_pages_free(p, None, None, 1, None) == ARG
    assert tqlib.tq_pages_free(p, P16, None, -1, None) == ARG
    assert tqlib.tq_pages_free(p, None, None, 0, None) == 0
    L = tb.make_layout(128, 32, 3)
    fork = lambda views=None, n_c=0, H=0, n=1, par=P16, ws=P16, nb=1 << 20: tqlib.tq_pages_fork(  # noqa: E731
        p, views, n_c, H, par, P16, P16, P16, n, None, ws, nb, None)
    assert fork(n=5) == ARG            # more entries than sequences
    assert fork(n=-1) == ARG
    assert fork(par=None) == ARG
    assert fork(ws=None) == WORKSPACE
    assert fork(nb=16) == WORKSPACE
    assert fork(ws=P8) == ALIGN
    assert fork(n_c=-1) == ARG
    assert fork(n_c=1, H=2) == ARG     # caches missing
    view = lambda **kw: (tb.tq_kv_view * 1)(tb.tq_kv_view(*{**dict(codes=16, scales=16, qjl=None, rnorm=None, S=None,  # noqa: E731
                                                                      layout=L, table=None, page=0, pps=0), **kw}.values()))
    assert fork(views=view(), n_c=1, H=0) == ARG
    assert fork(views=view(codes=None), n_c=1, H=2) == ARG
    assert fork(views=view(scales=8), n_c=1, H=2) == ALIGN
    assert fork(views=view(layout=tb.make_layout(96, 32, 3)), n_c=1, H=2) == UNSUP
    assert fork(views=view(layout=tb.make_layout(128, 128, 2, qjl_m=128)), n_c=1, H=2) == ARG   # no sign bits
    assert tqlib.tq_pages_compact(p, None, 0, 0, None, None, 0, None) == WORKSPACE
    assert tqlib.tq_pages_compact(p, None, 0, 0, None, P8, 1 << 20, None) == ALIGN


def test_page_workspace_query(tqlib):
    nb = ctypes.c_size_t()
    assert tqlib.tq_pages_workspace_bytes(4, 32, 3, ctypes.byref(nb)) == 0 and nb.value > 0
    assert tqlib.tq_pages_workspace_bytes(0, 32, 3, ctypes.byref(nb)) == ARG
    assert tqlib.tq_pages_workspace_bytes(4, 0, 3, ctypes.byref(nb)) == ARG
    assert tqlib.tq_pages_workspace_bytes(4, 32, -1, ctypes.byref(nb)) == ARG
    assert tqlib.tq_pages_workspace_bytes(4, 32, 3, None) == ARG


def test_view_follows_the_table(tqlib):
    """The kept C view is built anew when the table is another one of the same
    storage, or the arrays are others."""
    import torch
    L = tb.make_layout(128, 32, 3)
    codes = torch.zeros(16, 2, 32, 48, dtype=torch.uint8)
    scales = torch.zeros(16, 2, 32, 4, dtype=torch.float16)
    table = torch.zeros(16, dtype=torch.int32)
    c = tb.PackedKV.of(L, codes, scales, page_table=table.view(2, 8))
    assert (c.view().pages_per_seq, c.view().page_size) == (8, 32)
    c.page_table = table.view(4, 4)
    assert c.view().pages_per_seq == 4
    c.page_table = table.view(2, 8)[:, :4]
    assert c.view().pages_per_seq == 8 and c.capacity == 128
    c.page_table = None
    assert c.view().pages_per_seq == 0 and not c.view().page_table
    c.codes = codes.clone()
    assert c.view().codes == c.codes.data_ptr()


def test_views_are_of_now_and_the_callers_own(tqlib):
    """A replaced or changed layout is in the next view, and a changed view is
    nobody else's."""
    import torch
    L = tb.make_layout(128, 32, 3)
    c = tb.PackedKV.of(L, torch.zeros(4, 2, 32, 48, dtype=torch.uint8), torch.zeros(4, 2, 32, 4, dtype=torch.float16))
    v = c.view()
    assert v.layout.sign_seed == 1
    c.layout = tb.make_layout(128, 32, 3, sign_seed=9)
    assert c.view().layout.sign_seed == 9 and v.layout.sign_seed == 1
    c.layout.norm_correct = 1
    assert c.view().layout.norm_correct == 1
    v = c.view()
    v.page_size, v.codes = 7, 16
    assert (c.view().page_size, c.view().codes) == (0, c.codes.data_ptr())


def test_calls_see_the_cache_as_it_is(tqlib):
    """What the C calls get equals a view of now after every kind of change,
    and is not the struct that view() hands out."""
    import torch
    L = tb.make_layout(128, 128, 2, qjl_m=128)
    cb, ns, qb = tb.tq_layout_sizes(L)
    z = lambda dt, *s: torch.zeros(s, dtype=dt)  # noqa: E731
    c = tb.PackedKV.of(L, z(torch.uint8, 4, 2, 32, cb), z(torch.float16, 4, 2, 32, ns), z(torch.uint8, 4, 2, 32, qb),
                       z(torch.float16, 4, 2, 32))

    def same():
        got = c._view_ref()._obj
        assert bytes(got) == bytes(c.view())
        v = c.view()
        v.codes = 16
        assert bytes(c._view_ref()._obj) == bytes(c.view()) != bytes(v)

    same()
    for name in ("codes", "scales", "qjl", "rnorm"):
        setattr(c, name, getattr(c, name).clone())
        same()
    c.S = torch.zeros(128, 128)
    same()
    c.layout = tb.make_layout(128, 128, 2, qjl_m=128, sign_seed=3)
    same()
    c.layout.norm_correct = 1
    same()
    table = torch.zeros(16, dtype=torch.int32)
    for t in (table.view(2, 8), table.view(4, 4), table.view(2, 8)[:, :3], table[8:].view(1, 8), None):
        c.page_table = t
        same()


def test_caches_are_copied_and_pickled(tqlib):
    """Also after a call has taken their views."""
    import copy
    import pickle

    import torch
    L = tb.make_layout(128, 32, 3)
    c = tb.PackedKV.of(L, torch.ones(4, 2, 32, 48, dtype=torch.uint8), torch.ones(4, 2, 32, 4, dtype=torch.float16))
    c._view_ref()
    for d in (copy.copy(c), copy.deepcopy(c), pickle.loads(pickle.dumps(c))):
        assert torch.equal(d.codes, c.codes) and bytes(d.layout) == bytes(c.layout)
        assert d._view_ref()._obj.codes == d.codes.data_ptr()


def test_page_table_rows_are_contiguous(tqlib):
    """Columns that lie apart are no table that the C side can read."""
    import torch
    L = tb.make_layout(128, 32, 3)
    table = torch.zeros(4, 8, dtype=torch.int32)
    c = tb.PackedKV.of(L, torch.zeros(16, 2, 32, 48, dtype=torch.uint8), torch.zeros(16, 2, 32, 4, dtype=torch.float16),
                       page_table=table[:, :4])
    assert c.view().pages_per_seq == 8
    for t in (table[:, ::2], table.t()):
        c.page_table = t
        for call in (c.view, c._view_ref, c._table_stride):
            with pytest.raises(ValueError):
                call()
    c.page_table = table[:, 3:4]
    assert (c.view().pages_per_seq, c.capacity) == (8, 32)
