"""Calls on a stream that is not the current one: what a call makes for itself
(outputs, fills, copies of strided inputs, workspaces) belongs to the stream
that its kernels run on."""
import types

import numpy as np
import pytest
import torch

from turboquant_kv_cache_gb300 import inputs

pytestmark = pytest.mark.gpu


@pytest.fixture
def made(monkeypatch):
    """The streams that were current when torch.empty, zeros and empty_like ran."""
    seen = []
    for name in ("empty", "zeros", "empty_like"):
        real = getattr(torch, name)

        def wrapped(*a, _real=real, **k):
            seen.append(torch.cuda.current_stream().cuda_stream)
            return _real(*a, **k)

        monkeypatch.setattr(torch, name, wrapped)
    return seen


def _held_back(call):
    """call(stream) on a side stream while the current stream is busy for some
    20 ms: what a call orders there comes too late."""
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(40_000_000)
    out = call(side)
    torch.cuda.synchronize()
    return out


def _rows(B=3, T=17, Hq=4, Hkv=2, d=64):
    wide = torch.from_numpy(inputs.gaussian((B, T + 3, (Hq + 2 * Hkv) * d), 1)).cuda()
    ang = np.arange(64)[:, None] * 1e4 ** (-np.arange(0, d, 2) / d)
    rope = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).cuda()
    return wide[:, :T], rope, (Hq, Hkv, d), torch.tensor([0, 5, 40], dtype=torch.int32, device="cuda")


def test_rows_on_another_stream(tqlib):
    """Zeroed outputs and the copy of a strided input (batches that lie further
    apart than their tokens need)."""
    from turboquant_kv_cache_gb300 import binding as tb
    x, rope, sizes, pos = _rows()
    assert not x.is_contiguous()
    want = tb.tq_qkv_norm_rope(x, *sizes, rope=rope, pos=pos)
    got = _held_back(lambda s: tb.tq_qkv_norm_rope(x, *sizes, rope=rope, pos=pos, stream=s))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def _attention(tb):
    L = tb.make_layout(128, 32, 3)
    mk = lambda lead, seed: tb.tq_quantize_kv(L, torch.from_numpy(inputs.gaussian(lead + (128,), seed)).cuda())  # noqa: E731
    q = torch.from_numpy(inputs.gaussian((3, 8, 128), 5)).cuda()
    return (mk((1, 2, 700), 1), mk((1, 2, 700), 2), mk((3, 2, 64), 3), mk((3, 2, 64), 4)), q


def test_shared_decode_on_another_stream(tqlib):
    from turboquant_kv_cache_gb300 import binding as tb
    caches, q = _attention(tb)
    want = tb.tq_decode_attn_shared(*caches, q)
    assert torch.equal(_held_back(lambda s: tb.tq_decode_attn_shared(*caches, q, stream=s)), want)


def test_pages_on_another_stream(tqlib):
    from turboquant_kv_cache_gb300 import binding as tb
    L = tb.make_layout(64, 32, 4)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    results = []
    for hold in (False, True):
        c = tb.PackedKV(L, (40, 2, 32))
        c.codes.view(-1).copy_(torch.arange(c.codes.numel(), device="cuda") % 251)
        c.scales.zero_()
        pool = tb.PagePool.new(4, 8, 40, 32, [c])
        entries = [i32(-1, -1), i32(0, 1), i32(0, 0), i32(200, 70)], [i32(0, 1), i32(2, 3), i32(77, 70), i32(90, 130)]
        gone = i32(0)

        def steps(s):
            a = tb.tq_pages_fork(pool, *entries[0], stream=s)
            b = tb.tq_pages_fork(pool, *entries[1], stream=s)
            tb.tq_pages_free(pool, gone, stream=s)
            return a, b, tb.tq_pages_compact(pool, stream=s)

        r = _held_back(steps) if hold else steps(None)
        results.append([*r, pool.page_table, pool.n_pages, pool.ref, c.codes])
    assert results[0][0].tolist() == [0, 10, 0, 0]
    n = results[0][4].tolist()
    for a, b in zip(results[0][:3] + results[0][4:], results[1][:3] + results[1][4:]):
        assert torch.equal(a, b)
    for i in range(4):
        assert torch.equal(results[0][3][i, :n[i]], results[1][3][i, :n[i]])


def test_what_new_calls_make_is_their_streams(tqlib, made):
    from turboquant_kv_cache_gb300 import binding as tb
    x, rope, sizes, pos = _rows()
    caches, q = _attention(tb)
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    pool = tb.PagePool.new(4, 8, 40, 32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for call in (lambda: tb.tq_qkv_norm_rope(x, *sizes, stream=side), lambda: tb.tq_qkv_norm_rope(x, *sizes, slot=pos, stream=side),
                 lambda: tb.tq_decode_attn_shared(*caches, q, stream=side),
                 lambda: tb.tq_pages_fork(pool, one, one, one, one, stream=side), lambda: tb.tq_pages_compact(pool, stream=side)):
        made.clear()
        call()
        assert len(made) >= 2 and set(made) == {side.cuda_stream}
    torch.cuda.synchronize()


def test_stream_of_another_device_is_refused(tqlib):
    from turboquant_kv_cache_gb300 import binding as tb
    x, rope, sizes, pos = _rows()
    caches, q = _attention(tb)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    outs = tb.tq_qkv_norm_rope(x, *sizes)
    far = types.SimpleNamespace(cuda_stream=0, device_index=q.get_device() + 1)
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        tb.tq_decode_attn_shared(*caches, q, workspace=ws, out=torch.empty_like(q), stream=far)
    with pytest.raises(ValueError):
        tb.tq_qkv_norm_rope(x.contiguous(), *sizes, q_out=outs[0], k_out=outs[1], v_out=outs[2], stream=far)
    with pytest.raises(ValueError):
        tb.tq_pages_free(tb.PagePool.new(4, 8, 40, 32), one, stream=far)


def _codec(tb):
    """Inputs that the calls copy before their kernels read them."""
    L = tb.make_layout(128, 32, 3)
    x = torch.from_numpy(inputs.gaussian((2, 40, 3, 128), 21)).cuda().transpose(1, 2)       # [2, 3, 40, 128], strided
    pos = torch.tensor([[3, 9], [0, 9]], dtype=torch.int32, device="cuda")[:, 0]
    q = torch.from_numpy(inputs.gaussian((2, 6, 128), 22)).cuda()
    return L, x, pos, q


def test_codec_on_another_stream(tqlib):
    from turboquant_kv_cache_gb300 import binding as tb
    L, x, pos, q = _codec(tb)

    def append(s):
        c = tb.PackedKV(L, (2, 3, 64))
        c.codes.zero_()
        c.scales.zero_()
        if s is not None:
            torch.cuda.synchronize()     # the cache is filled before the side stream has it
            torch.cuda._sleep(40_000_000)
        return tb.tq_append_kv(c, x, pos, stream=s)

    for call in (lambda s: tb.tq_quantize_kv(L, x, stream=s), append):
        want, got = call(None), _held_back(call)
        assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
    want, got = (f(lambda s: tb.tq_polar_quantize(x, 3, stream=s)) for f in (lambda c: c(None), _held_back))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    K = tb.tq_quantize_kv(L, x)
    # a window whose rows lie apart
    win = torch.from_numpy(inputs.gaussian((2, 7, 3, 128), 23)).cuda().transpose(1, 2)
    call = lambda s: tb.tq_decode_attn_window(K, K, q, win, win, stream=s)  # noqa: E731
    assert torch.equal(_held_back(call), call(None))


def test_what_the_other_calls_make_is_their_streams(tqlib, made):
    from turboquant_kv_cache_gb300 import binding as tb
    L, x, pos, q = _codec(tb)
    K = tb.tq_quantize_kv(L, x)
    blocks = tb.tq_to_blocks(K)
    codes, radius = tb.tq_polar_quantize(x, 3)
    win = torch.zeros(2, 3, 8, 128, dtype=torch.float16, device="cuda")
    q4 = q[:, :, None].expand(-1, -1, 5, -1).contiguous()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for call in (lambda: tb.tq_quantize_kv(L, x, stream=side), lambda: tb.tq_dequantize_kv(K, stream=side),
                 lambda: tb.tq_decode_attn(K, K, q, stream=side), lambda: tb.tq_decode_attn_static(K, K, q, stream=side),
                 lambda: tb.tq_decode_attn_window(K, K, q, win, win, stream=side), lambda: tb.tq_to_blocks(K, stream=side),
                 lambda: tb.tq_from_blocks(L, blocks, stream=side),
                 lambda: tb.tq_decode_attn_blocks(L, blocks, L, blocks, q, stream=side),
                 lambda: tb.tq_polar_quantize(x, 3, stream=side), lambda: tb.tq_polar_dequantize(codes, radius, 128, 3, stream=side),
                 lambda: tb.tq_prefill_attn(K, K, q4, 40, stream=side)):
        made.clear()
        call()
        assert made and set(made) == {side.cuda_stream}
    torch.cuda.synchronize()
