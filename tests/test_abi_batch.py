"""Argument checks of the ragged-batch and beam-search calls: every refusal
happens on the host, so none of this needs a GPU."""
import ctypes

import pytest

from turboquant_kv_cache_gb300 import binding as tb

P16, P8, P4, P2, P1 = (ctypes.c_void_p(1 << 20 | k) for k in (0, 8, 4, 2, 1))
OK, ARG, UNSUP, ALIGN, WORKSPACE = 0, -1, -2, -3, -4


def _slots(lib, new=P16, have=P16, B=3, cap=256, table=P16, page=64, pps=4, n=10, start=P16, seq=P16, pos=P16, slot=P16,
           rlen=P16, rtab=None, rpages=0, result=P16):
    return lib.tq_batch_slots(new, have, B, cap, table, page, pps, n, start, seq, pos, slot, rlen, rtab, rpages, result, None)


@pytest.mark.parametrize("kw,status", [
    (dict(new=None), ARG), (dict(start=None), ARG), (dict(pos=None), ARG), (dict(slot=None), ARG), (dict(B=0), ARG),
    (dict(n=-1), ARG), (dict(cap=0), ARG), (dict(cap=257), ARG), (dict(page=48), ARG), (dict(page=0), ARG), (dict(pps=0), ARG),
    (dict(rtab=P16, rpages=5), ARG), (dict(rtab=P16, rpages=0), ARG), (dict(rpages=-1), ARG),
    (dict(table=None, rtab=P16, rpages=1), ARG), (dict(table=None, cap=2**31 - 64), UNSUP), (dict(B=(1 << 20) + 1), UNSUP),
    (dict(new=P2), ALIGN), (dict(have=P2), ALIGN), (dict(table=P2), ALIGN), (dict(start=P2), ALIGN), (dict(rtab=P2, rpages=1), ALIGN),
    (dict(result=P2), ALIGN), (dict(seq=P8), ALIGN), (dict(pos=P4), ALIGN), (dict(slot=P8), ALIGN), (dict(rlen=P8), ALIGN),
])
def test_batch_slots_refusals(tqlib, kw, status):
    assert _slots(tqlib, **kw) == status


def _append(lib, L=None, x=P16, dt=0, n=5, H=2, stride=128, slot=P16, spp=64, ns=640, codes=P16, scales=P16):
    L = L or tb.make_layout(128, 32, 3)
    return lib.tq_append_kv_slots(ctypes.byref(L), x, dt, n, H, stride, slot, spp, ns, None, codes, scales, None, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), ARG), (dict(H=-1), ARG), (dict(spp=0), ARG), (dict(spp=-1), ARG), (dict(ns=-1), ARG), (dict(ns=100), ARG),
    (dict(slot=None), ARG), (dict(x=None), ARG), (dict(codes=None), ARG), (dict(scales=None), ARG), (dict(stride=127), ARG),
    (dict(dt=2), ARG), (dict(slot=P4), ALIGN), (dict(x=P8), ALIGN), (dict(codes=P8), ALIGN), (dict(stride=129), ALIGN),
    (dict(L=tb.make_layout(96, 32, 3)), UNSUP), (dict(L=tb.make_layout(128, 128, 2, qjl_m=64)), ARG), (dict(n=0), OK), (dict(H=0), OK),
])
def test_append_slots_refusals(tqlib, kw, status):
    assert _append(tqlib, **kw) == status


def _beam(lib, x=P16, dt=1, B=2, W=4, V=1000, stride=None, scores=P16, done=P16, eos=2, n=4, keep=0, os=P16, op=P16, ot=P16, od=P16,
          ws=P16, nbytes=1 << 24):
    return lib.tq_beam_select(x, dt, B, W, V, V if stride is None else stride, scores, done, eos, n, keep, os, op, ot, od, ws, nbytes,
                              None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), ARG), (dict(os=None), ARG), (dict(op=None), ARG), (dict(ot=None), ARG), (dict(dt=2), ARG), (dict(B=0), ARG),
    (dict(W=0), ARG), (dict(V=0), ARG), (dict(n=0), ARG), (dict(stride=999), ARG), (dict(eos=1000), ARG), (dict(eos=-2), ARG),
    (dict(eos=-1), ARG),                      # finished beams need the token that finished them
    (dict(keep=1, n=3), ARG), (dict(W=1, V=3, n=4, stride=3), ARG), (dict(W=65), UNSUP), (dict(n=65), UNSUP),
    (dict(V=1 << 26), UNSUP), (dict(B=1 << 30, W=64), UNSUP),
    (dict(x=P2), ALIGN), (dict(x=P1, dt=0), ALIGN), (dict(scores=P2), ALIGN), (dict(os=P2), ALIGN), (dict(op=P2), ALIGN),
    (dict(ot=P2), ALIGN), (dict(ws=P8), ALIGN), (dict(ws=None), WORKSPACE), (dict(nbytes=64), WORKSPACE),
])
def test_beam_refusals(tqlib, kw, status):
    assert _beam(tqlib, **kw) == status


def test_beam_workspace_query(tqlib):
    nb = ctypes.c_size_t()
    q = lambda *a: tqlib.tq_beam_workspace_bytes(*a, ctypes.byref(nb))  # noqa: E731
    assert q(4, 4, 32000, 8) == OK and nb.value > 0
    assert q(4, 4, 32000, 65) == UNSUP and q(4, 0, 32000, 4) == ARG and q(1, 1, 3, 4) == ARG
    assert tqlib.tq_beam_workspace_bytes(4, 4, 32000, 8, None) == ARG


def _states(lib, n=1, n_seqs=8, W=4, parent=P16, **kw):
    a = dict(data=1 << 20, len=1 << 21, cap=100, heads=2, bytes=48)
    a.update(kw)
    s = (tb.tq_state_array * 2)(tb.tq_state_array(**a), tb.tq_state_array(**a))
    return lib.tq_states_reorder(s, n, n_seqs, W, parent, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), ARG), (dict(n_seqs=-4), ARG), (dict(W=0), ARG), (dict(n_seqs=6), ARG), (dict(parent=None), ARG),
    (dict(data=None), ARG), (dict(cap=-1), ARG), (dict(heads=0), ARG), (dict(bytes=0), ARG), (dict(W=65, n_seqs=65), UNSUP),
    (dict(cap=1 << 31), UNSUP), (dict(heads=1 << 20), UNSUP), (dict(parent=P2), ALIGN), (dict(len=(1 << 21) + 2), ALIGN),
    (dict(n=0), OK), (dict(n_seqs=0), OK), (dict(W=1), OK),
])
def test_states_refusals(tqlib, kw, status):
    assert _states(tqlib, **kw) == status
    assert tqlib.tq_states_reorder(None, 1, 8, 4, P16, None) == ARG


def _tables(lib, pool=(1 << 20, 1 << 20, 1 << 20, 16, 8, 64, 64), parent=P16, seqs=None, n=8, ws=P16, nbytes=1 << 20):
    p = tb.tq_page_pool(*pool) if pool else None
    return lib.tq_pages_reorder(ctypes.byref(p) if p else None, parent, seqs, n, None, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(pool=None), ARG), (dict(pool=(None, 1 << 20, 1 << 20, 16, 8, 64, 64)), ARG),
    (dict(pool=(1 << 20, 1 << 20, 1 << 20, 16, 8, 64, 48)), ARG), (dict(n=-1), ARG), (dict(n=17), ARG), (dict(parent=None), ARG),
    (dict(ws=None), WORKSPACE), (dict(nbytes=100), WORKSPACE), (dict(ws=P8), ALIGN),
    (dict(pool=(1 << 20, 1 << 20, 1 << 20, 16, 1 << 21, 64, 64)), UNSUP),
])
def test_tables_refusals(tqlib, kw, status):
    assert _tables(tqlib, **kw) == status


def test_tables_workspace_query(tqlib):
    nb = ctypes.c_size_t()
    assert tqlib.tq_pages_reorder_workspace_bytes(16, 8, 8, ctypes.byref(nb)) == OK and nb.value >= 4 * 8 * 8
    assert tqlib.tq_pages_reorder_workspace_bytes(0, 8, 8, ctypes.byref(nb)) == ARG
    assert tqlib.tq_pages_reorder_workspace_bytes(16, 8, -1, ctypes.byref(nb)) == ARG
    assert tqlib.tq_pages_reorder_workspace_bytes(16, 8, 8, None) == ARG
