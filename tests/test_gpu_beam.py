"""Beam selection against scores in 64 bits.

Bound of a score's error: the logits are exact, so it is that of lse plus half
a step of the fp32 result.  A term exp(x - m) is off by 2^-22 (ex2.approx) and by
the roundings of x - m and of its product with log2 e, 2^-23 |x - m| together;
weighted with the terms themselves the mean of |x - m| is at most log V.  A
thread adds up less than 128 terms before it keeps what a sum rounds off, the
parts of a row are some ten more sums and one more exp: (4 + 2 log V) + 140 + (4 + 2 log V) in units of 2^-24."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def lse_bound(V):
    return (148 + 4 * np.log(V)) * 2.0 ** -24


def reference(x, scores, n, done=None, eos=-1):
    """Scores [B, W V] in 64 bits and the places of the n best, ties by place."""
    x = np.nan_to_num(x.astype(np.float64), nan=-np.inf, posinf=float(np.finfo(np.float32).max), neginf=-np.inf)
    s = np.nan_to_num(scores.astype(np.float64), nan=-np.inf, posinf=float(np.finfo(np.float32).max), neginf=-np.inf)
    B, W, V = x.shape
    m = x.max(-1, keepdims=True)
    m0 = np.where(np.isinf(m), 0.0, m)
    with np.errstate(divide="ignore", invalid="ignore"):
        # the difference first: next to a mask's lowest value the sum of m and the logarithm is m
        lp = (x - m0) - np.log(np.exp(x - m0).sum(-1, keepdims=True))
    lp = np.where(np.isinf(x), -np.inf, lp)
    if done is not None:
        lp = np.where(done.astype(bool)[..., None], np.where(np.arange(V) == eos, 0.0, -np.inf), lp)
    full = (np.where(np.isinf(s), -np.inf, s)[..., None] + lp).reshape(B, W * V)
    full = np.where(np.repeat(np.isinf(s), V, axis=-1).reshape(B, W * V), -np.inf, full)
    # where 64 bits do not tell two candidates apart, what they round off does: the exact sum is full + rest
    big, lp2 = np.repeat(np.where(np.isinf(s), 0.0, s), V, axis=-1).reshape(B, W * V), lp.reshape(B, W * V)
    with np.errstate(invalid="ignore"):
        part = full - big
        rest = (big - (full - part)) + (lp2 - part)
    rest = np.where(np.isfinite(rest), rest, 0.0)
    return full, np.stack([np.lexsort((np.arange(W * V), -r, -f))[:n] for f, r in zip(full, rest)])


def placed(order, V, W):
    """What keep_place makes of the places by score."""
    out = np.empty_like(order)
    for b, row in enumerate(order):
        place, rest = {}, []
        for f in row:
            w = f // V
            if w in place:
                rest.append(f)
            else:
                place[w] = f
        for k in range(W):
            if k not in place:
                place[k] = rest.pop(0)
        out[b] = [place[k] for k in range(W)]
    return out


def check(x, scores, n, out, done=None, eos=-1, keep=False):
    V, W = x.shape[2], x.shape[1]
    host = x.float().cpu().numpy()
    s = scores.cpu().numpy() if scores is not None else np.zeros(host.shape[:2])
    d = done.cpu().numpy() if done is not None else None
    full, order = reference(host, s, n, d, eos)
    got_s, parent, token, got_done = (t.cpu().numpy() for t in out)
    B = host.shape[0]
    flat = (parent - np.arange(B)[:, None] * W).astype(np.int64) * V + token
    tol = lse_bound(V)
    if keep:
        order = placed(order, V, W)
    want = np.take_along_axis(full, order, -1)
    mine = np.take_along_axis(full, flat, -1)
    near = (flat != order) & (np.abs(np.where(np.isinf(want), -1e30, want) - np.where(np.isinf(mine), -1e30, mine)) <= 2 * tol)
    assert ((flat == order) | near).all() and near.sum() <= 2, (flat[~near & (flat != order)], order[~near & (flat != order)])
    assert (np.isinf(mine) == np.isinf(got_s)).all()
    fine = ~np.isinf(mine)
    err = np.abs(got_s.astype(np.float64)[fine] - mine[fine])
    assert (err <= tol + np.abs(mine[fine]) * 2.0 ** -24).all(), err.max()
    ended = (d[np.arange(B)[:, None], flat // V].astype(bool) if d is not None else False) | (token == eos)
    assert (got_done.astype(bool) == ended).all()
    for b in range(B):
        assert len(set(flat[b].tolist())) == n


SIZES = [  # B, W, V, n_out
    (1, 1, 1, 1), (1, 1, 5, 5), (2, 3, 2, 6), (1, 4, 37, 8), (3, 5, 1000, 5), (2, 4, 32000, 8), (1, 1, 50021, 16), (7, 5, 4097, 5),
    (1, 64, 700, 64), (2, 16, 30011, 32), (40, 8, 8191, 8), (1, 2, 200003, 64), (5, 1, 128256, 64), (600, 2, 3001, 2), (1, 64, 33, 64), (100, 4, 30011, 4), (37, 5, 50021, 12), (9, 7, 128256, 40)]


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("B,W,V,n", SIZES)
def test_beam_select(tqlib, B, W, V, n, f32):
    from turboquant_kv_cache_gb300 import binding as tb
    g = torch.Generator(device="cuda").manual_seed(B * W + V)
    x = 3 * torch.randn(B, W, V, generator=g, device="cuda")
    x = x if f32 else x.half()
    scores = -5 * torch.rand(B, W, generator=g, device="cuda")
    check(x, scores, n, tb.tq_beam_select(x, scores, n_out=n), )
    check(x, None, n, tb.tq_beam_select(x, None, n_out=n))
    if V > 2:
        done = (torch.rand(B, W, generator=g, device="cuda") < 0.4).to(torch.uint8)
        check(x, scores, n, tb.tq_beam_select(x, scores, n_out=n, done=done, eos=V // 2), done, V // 2)
    if W * V >= W:
        check(x, scores, W, tb.tq_beam_select(x, scores, keep_place=True, eos=0), eos=0, keep=True)


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("V", [3000, 50021])
@pytest.mark.parametrize("mask", ["inf", "lowest", "all", "same", "few_values", "hot_threads", "sorted", "nan_inf"])
def test_beam_select_masks_and_ties(tqlib, mask, V, f32):
    """Shut-out tokens by -inf and by the type's lowest value, rows that leave
    nothing, repeated values, large values gathered where one thread has them,
    NaN and infinities."""
    from turboquant_kv_cache_gb300 import binding as tb
    B, W = 3, 5
    g = torch.Generator(device="cuda").manual_seed(V)
    x = 2 * torch.randn(B, W, V, generator=g, device="cuda")
    x = x if f32 else x.half()
    low = torch.finfo(x.dtype).min
    some = torch.rand(B, W, V, generator=g, device="cuda")
    if mask in ("inf", "lowest"):
        v = -float("inf") if mask == "inf" else low
        x[some > 9 / V] = v
        x[0, 1] = v                       # nothing left in one row
        x[1] = v                          # nor in a whole request
    elif mask == "all":
        x[:] = -float("inf")
    elif mask == "same":
        x[:] = 1.25
    elif mask == "few_values":
        x = x.round().clamp_max(3)        # many share the largest value
    elif mask == "hot_threads":
        x[:, :, :512] += 40               # every large value at the row's start
        x[:, 2, 700:1500] += 60
    elif mask == "sorted":
        x = x.sort(-1, descending=True).values
    else:
        x[some < 0.01] = float("nan")
        x[0, 0, 7] = float("inf")
        x[0, 3, ::5] = float("inf")
        x[1, 2] = float("nan")
        x[2, 1, 3] = -float("inf")
    scores = -torch.rand(B, W, generator=g, device="cuda")
    scores[2, 1:] = -float("inf")         # a first step: one beam lives
    for n in (1, W, 2 * W, 64):
        check(x, scores, n, tb.tq_beam_select(x, scores, n_out=n))
    check(x, scores, W, tb.tq_beam_select(x, scores, keep_place=True), keep=True)
    scores[:] = -float("inf")
    check(x, scores, W, tb.tq_beam_select(x, scores))
    scores[0, 0], scores[0, 1], scores[1, 0] = float("nan"), 0.0, 3e38
    done = torch.zeros(B, W, dtype=torch.bool, device="cuda")
    done[0, 0] = done[1, 4] = done[2, 2] = True
    check(x, scores, 2 * W, tb.tq_beam_select(x, scores, n_out=2 * W, done=done, eos=1), done, 1)


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("mask", ["inf", "lowest", "same", "few_values", "sorted", "rising", "first_inf", "first_lowest", "few_first",
                                  "last_hot", "late_nan", "late_inf", "huge"])
def test_beam_select_streamed_rows(tqlib, mask, f32):
    """Rows long and many enough that a CTA streams several parts: what the first
    part says of the rest is wrong in each of these, or leaves nothing."""
    from turboquant_kv_cache_gb300 import binding as tb
    B, W, V = 31, 5, 20011
    g = torch.Generator(device="cuda").manual_seed(17)
    x = 2 * torch.randn(B, W, V, generator=g, device="cuda")
    x = x if f32 else x.half()
    low = torch.finfo(x.dtype).min
    some = torch.rand(B, W, V, generator=g, device="cuda")
    if mask in ("inf", "lowest"):
        v = -float("inf") if mask == "inf" else low
        x[some > 20 / V] = v
        x[0, 1] = x[1] = v
    elif mask == "same":
        x[:] = -3.5
    elif mask == "few_values":
        x = x.round().clamp_max(3)
    elif mask in ("sorted", "rising"):
        x = x.sort(-1, descending=mask == "sorted").values
    elif mask in ("first_inf", "first_lowest"):
        x[:, :, :9000] = -float("inf") if mask == "first_inf" else low
    elif mask == "few_first":
        x[:, :, :4300] = -float("inf")
        x[:, 1, 77] = x[:, 2, 4000] = 1.0
    elif mask == "last_hot":
        x[:, :, -40:] += 150              # e^150 is out of the range of 32 bits
        x[:, 3, 12000] = 90
    elif mask == "late_nan":
        x[:, :, 15000::7] = float("nan")
    elif mask == "late_inf":
        x[:, 1, 17000] = x[:, 2, 5000] = x[:, 2, 19000] = float("inf")
    else:
        x = (x.float() * (1e36 if f32 else 3e4)).to(x.dtype)
    scores = -torch.rand(B, W, generator=g, device="cuda")
    scores[2, 1:] = -float("inf")
    for n in (W, 48):
        check(x, scores, n, tb.tq_beam_select(x, scores, n_out=n))


@pytest.mark.parametrize("M,W,V", [(64, 64, 200000), (64, 1, 200000), (50, 2, 70000)])
def test_beam_select_full_lists(tqlib, M, W, V):
    """More candidates above the bounds than the lists hold: each row's largest
    values beside each other, so that single parts and threads have them."""
    from turboquant_kv_cache_gb300 import binding as tb
    for f32 in (True, False):
        x = torch.zeros(1, W, V, device="cuda")
        x[:] = torch.linspace(-1, 1, V, device="cuda")
        g = torch.Generator(device="cuda").manual_seed(M)
        for w in range(W):
            at = 1000 * (w % 7) + torch.arange(3000, device="cuda")
            x[0, w, at] = 20 + torch.rand(3000, generator=g, device="cuda")
        x[0, :, 128 * 4 * 3::128 * 8] += 30       # one thread's places
        x = x if f32 else x.half()
        scores = -torch.rand(1, W, generator=g, device="cuda")
        check(x, scores, M, tb.tq_beam_select(x, scores, n_out=M))


def test_beam_select_strides_and_outputs(tqlib):
    """Rows that start anywhere, padded rows, a transposed batch, outputs in
    place of the inputs, an expanded tensor, a captured replay, another stream."""
    from turboquant_kv_cache_gb300 import binding as tb
    g = torch.Generator(device="cuda").manual_seed(3)
    B, W, V = 2, 3, 5003
    scores = -torch.rand(B, W, generator=g, device="cuda")
    for dt in (torch.float32, torch.float16):
        flat = (3 * torch.randn(B * W * (V + 9) + 64, generator=g, device="cuda")).to(dt)
        for off in (0, 1, 3, 7):
            for pad in (0, 1, 8):
                x = flat[off:off + B * W * (V + pad)].view(B, W, V + pad)[:, :, :V]
                check(x, scores, W, tb.tq_beam_select(x, scores))
    x = torch.randn(W, B, V, generator=g, device="cuda")
    check(x.transpose(0, 1), scores, W, tb.tq_beam_select(x.transpose(0, 1), scores))
    e = torch.randn(1, 1, V, generator=g, device="cuda").expand(B, W, V)
    check(e, scores, W, tb.tq_beam_select(e, scores))
    x = torch.randn(B, W, V, generator=g, device="cuda")
    done = torch.zeros(B, W, dtype=torch.uint8, device="cuda")
    s0, d0 = scores.clone(), done.clone()
    ids = torch.empty(2, B, W, dtype=torch.int32, device="cuda")
    ws = torch.empty(tb.tq_beam_workspace_bytes(B, W, V, W), dtype=torch.uint8, device="cuda")
    call = lambda: tb.tq_beam_select(x, scores, done=done, eos=7, workspace=ws, out=(scores, ids[0], ids[1], done))  # noqa: E731
    call()
    check(x, s0, W, (scores, ids[0], ids[1], done), d0, 7)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in range(3):
        x.copy_(2 * torch.randn(B, W, V, generator=g, device="cuda"))
        x[0, k, 7] = 30.0
        s0, d0 = scores.clone(), done.clone()
        graph.replay()
        torch.cuda.synchronize()
        check(x, s0, W, (scores, ids[0], ids[1], done), d0, 7)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = tb.tq_beam_select(x, s0, stream=side)
    side.synchronize()
    check(x, s0, W, out)


def test_beam_select_long_rows(tqlib):
    """Rows of millions of tokens: the bound does not grow with their length, and
    the best are found at both ends."""
    from turboquant_kv_cache_gb300 import binding as tb
    V = 5_000_011
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(1, 2, V, generator=g, device="cuda")
    x[0, 0, 0] = x[0, 1, V - 1] = 9.0
    scores = torch.tensor([[-1.0, -1.25]], device="cuda")
    for t in (x, x.half()):
        check(t, scores, 5, tb.tq_beam_select(t, scores, n_out=5))


def test_beam_select_long_offsets(tqlib):
    """Rows that lie behind 2^31 logits."""
    from turboquant_kv_cache_gb300 import binding as tb
    stride = (1 << 31) // 3 + 5
    big = torch.empty(3 * stride + 4096, dtype=torch.float16, device="cuda")
    x = big.as_strided((4, 1, 4001), (stride, stride, 1))
    x.copy_(torch.randn(4, 1, 4001, device="cuda"))
    scores = torch.zeros(4, 1, device="cuda")
    check(x, scores, 9, tb.tq_beam_select(x, scores, n_out=9))


def test_beam_select_refusals(tqlib):
    from turboquant_kv_cache_gb300 import binding as tb
    x = torch.randn(2, 3, 100, device="cuda")
    f = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    for kw in (dict(scores=f(2, 4)), dict(scores=f(2, 3, dt=torch.float16)), dict(scores=f(3, 2).t()), dict(done=f(2, 3)),
               dict(done=f(2, 4, dt=torch.uint8)), dict(out=(f(2, 3),) * 4), dict(out=(f(2, 3),) * 3),
               dict(workspace=torch.empty(100, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            tb.tq_beam_select(x, **kw)
    for kw in (dict(n_out=65), dict(n_out=4, keep_place=True), dict(done=f(2, 3, dt=torch.uint8)), dict(eos=100),
               dict(workspace=f(16))):
        with pytest.raises(tb.TQError):
            tb.tq_beam_select(x, **kw)
    for bad in (x[0], x.cpu(), x.transpose(1, 2)):
        with pytest.raises(ValueError):
            tb.tq_beam_select(bad)
    with pytest.raises(TypeError):
        tb.tq_beam_select(x.double())
