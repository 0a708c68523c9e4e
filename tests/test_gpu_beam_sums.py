"""Beam selection: the sum of a row's exponentials where its terms' reference matters.

A row of largest logit m has lse = m + log S, S = sum exp(x - m), and S is 1 for
the largest logit itself, exactly: exp(0) is."""
import numpy as np
import pytest
import torch

from test_gpu_beam import check

pytestmark = pytest.mark.gpu

# maxima whose product with log2 e is rounded by 126 and more (the first three), by less, and by more than 32 bits hold
LARGE = [2.06e9, 2.68e9, 6.19e9, 1e3, 3e6, 1.7e7, 1e9, 1e12, 1e20, 1e36, 2.5e38]


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("V", [1, 5, 3000])
def test_beam_select_large_logits(tqlib, V, sign):
    """Finite logits give finite scores, however large: a row of one token scores 0."""
    from turboquant_kv_cache_gb300 import binding as tb
    g = torch.Generator(device="cuda").manual_seed(V)
    top = sign * torch.tensor(LARGE, device="cuda")
    x = top.view(-1, 1, 1) - top.abs().view(-1, 1, 1) * 0.3 * torch.rand(len(LARGE), 2, V, generator=g, device="cuda")
    x[:, :, V // 2] = top.view(-1, 1)
    n = min(4, 2 * V)
    out = tb.tq_beam_select(x, n_out=n)
    check(x, None, n, out)
    if V == 1:
        assert (out[0] == 0).all()
    else:   # where no other logit of a row is within 40 of its largest, S is 1 and the score 0
        first, second = x.double().topk(2, -1).values.unbind(-1)
        alone = (first - second > 40).all(-1)
        assert alone.sum() >= 6 and torch.isfinite(out[0]).all() and (out[0][alone][:, :2] == 0).all()


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("at", [77, 9000, 20010])
def test_beam_select_large_logits_streamed(tqlib, at, sign):
    """The same where a CTA goes through several parts of a row, the maximum in its
    first part, in a later one and in the last place."""
    from turboquant_kv_cache_gb300 import binding as tb
    B, W, V = 3 * len(LARGE), 5, 20011
    g = torch.Generator(device="cuda").manual_seed(at)
    top = (sign * torch.tensor(LARGE, device="cuda")).repeat(3).view(-1, 1)
    x = top.unsqueeze(-1) - top.abs().unsqueeze(-1) * (0.1 + 0.2 * torch.rand(B, W, V, generator=g, device="cuda"))
    x[:, :, at] = top
    scores = -torch.rand(B, W, generator=g, device="cuda")
    out = tb.tq_beam_select(x, scores, n_out=W)
    check(x, scores, W, out)
    assert torch.equal(out[0], scores.sort(-1, descending=True).values) and (out[2] == at).all()


U = 2.0 ** -24   # half a step at 1: what a rounding to 32 bits is off by, at most, of its result


def _sparse(B, V, f32, gap, seed):
    """Rows of two tokens, 0 among the first 4000 and a larger one by gap to gap + 1
    behind them; all others have no weight in 32 bits (exp(-200))."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.full((B, V), -200.0, device="cuda")
    r = torch.arange(B, device="cuda")
    first = torch.randint(0, 4000, (B,), generator=g, device="cuda")
    last = torch.randint(4200, V, (B,), generator=g, device="cuda")
    last[0], last[-1] = V - 1, 4200
    x[r, first] = 0.0
    x[r, last] = gap + torch.rand(B, generator=g, device="cuda")
    return (x if f32 else x.half()), first, last


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("gap", [1, 5, 10, 20, 40, 60])
@pytest.mark.parametrize("B", [800, 200, 3])
def test_beam_select_late_maximum(tqlib, B, gap, f32):
    """The first logits say little of the row's largest, as where a trained model is
    sure of a token (a CTA for a row, for a few parts of one, for each part).

    S = 1 + exp(-g): the one is exact, the other off by a step and a half in its
    change of reference (expf a step, a product), their sum by a rounding, and the
    logarithm, below 0.32, by a step of its own (logf)."""
    from turboquant_kv_cache_gb300 import binding as tb
    V = 20011
    x, first, last = _sparse(B, V, f32, gap, B + gap)
    score, parent, token, _ = tb.tq_beam_select(x.unsqueeze(1), n_out=2)
    assert torch.equal(token[:, 0].long(), last) and torch.equal(token[:, 1].long(), first)
    g = x.double()[torch.arange(B, device="cuda"), last]
    log_s = torch.log1p(torch.exp(-g))
    tol = U * (1 + 3 * torch.exp(-g)) + 2 * U * log_s
    for k, want in enumerate((-log_s, -g - log_s)):
        err = (score[:, k].double() - want).abs()
        assert (err <= tol + U * want.abs()).all(), (k, (err - U * want.abs()).max().item())


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("gap", [30, 60])
def test_beam_select_sure_rows(tqlib, gap, f32):
    """The same with ordinary logits around: what they add to S is below half a step
    of 1, so the best score is the beam's own."""
    from turboquant_kv_cache_gb300 import binding as tb
    B, W, V = 160, 5, 20011
    g = torch.Generator(device="cuda").manual_seed(gap)
    x = 2 * torch.randn(B, W, V, generator=g, device="cuda")
    at = torch.randint(4200, V, (B, W, 1), generator=g, device="cuda")
    x.scatter_(2, at, x.amax(-1, keepdim=True) + gap + torch.rand(B, W, 1, generator=g, device="cuda"))
    x = x if f32 else x.half()
    d = x.double()
    assert ((torch.logsumexp(d, -1) - d.amax(-1)) < U / 2).all()
    scores = -5 * torch.rand(B, W, generator=g, device="cuda")
    out = tb.tq_beam_select(x, scores, n_out=W)
    check(x, scores, W, out)
    want, order = scores.sort(-1, descending=True)
    assert torch.equal(out[0], want) and torch.equal(out[2].long(), at.squeeze(-1).gather(1, order))


@pytest.mark.parametrize("f32", [True, False])
def test_beam_select_orders_rows_of_different_gaps(tqlib, f32):
    """Beams whose scores differ by 3e-7, each sure of its token by another amount:
    S is 1 for all (gaps from 20 on), so the beams' own scores order the candidates."""
    from turboquant_kv_cache_gb300 import binding as tb
    B, W, V = 160, 5, 20011
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.cat([_sparse(B, V, f32, gap, gap)[0].unsqueeze(1) for gap in (20, 30, 40, 50, 60)], 1)
    x = x[:, torch.randperm(W, generator=g, device="cuda")].contiguous()
    place = torch.rand(B, W, generator=g, device="cuda").argsort(-1)
    scores = -3e-7 * place
    out = tb.tq_beam_select(x, scores, n_out=W)
    rows = torch.arange(B, device="cuda")[:, None] * W + place.argsort(-1)
    assert torch.equal(out[1].long(), rows)
    assert (out[0].double() - scores.double().sort(-1, descending=True).values).abs().max() <= 2.1e-9 + 13e-7 * U


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("B", [800, 200, 3])
def test_beam_select_rising_maxima(tqlib, B, f32):
    """A row's largest logit replaced again and again, by steps of 1: sixteen terms
    are added up in some order and change their reference, the sum with them
    (a step and a half of a third of it each time): 15 + 3.4 roundings, and the
    logarithm of 1.58 with its own step."""
    from turboquant_kv_cache_gb300 import binding as tb
    V = 20011
    x = torch.full((B, 1, V), -200.0, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(B)
    for k in range(16):
        at = torch.randint(1200 * k, 1200 * (k + 1), (B, 1, 1), generator=g, device="cuda")
        x.scatter_(2, at, float(k))
    x = x if f32 else x.half()
    score = tb.tq_beam_select(x, n_out=16)[0].double()
    want = torch.arange(15, -1, -1, device="cuda").double()
    want = want - torch.logsumexp(want, 0)
    assert ((score - want).abs() <= 19 * U + U + U * want.abs()).all(), (score - want).abs().max()


@pytest.mark.parametrize("W,score,size", [(1, 1e30, 1e-10), (3, 1e30, 1e-10), (2, -3e38, 1e-10), (1, 0.0, 1e-19), (2, -4.5, 1e-19)])
def test_beam_select_equal_scores_of_different_logits(tqlib, W, score, size):
    """Logits whose differences a score does not hold: with a range of 2 size around 0
    they are below half a step of a pair of floats (2^-48 of the score, or 2^-24 of
    lse = log V where the score takes the first of the pair).  All candidates are equal then,
    those of the lower beam come first and of one beam the higher logits, wherever in
    the row they are; more of them than the list takes."""
    from turboquant_kv_cache_gb300 import binding as tb
    V, M = 128256, 64
    g = torch.Generator(device="cuda").manual_seed(W)
    x = size * (2 * torch.rand(1, W, V, generator=g, device="cuda") - 1)
    out = tb.tq_beam_select(x, torch.full((1, W), score, device="cuda"), n_out=M)
    order = np.lexsort((np.arange(V), -x[0, 0].double().cpu().numpy()))[:M]
    assert (out[1] == 0).all() and out[2][0].tolist() == order.tolist()


@pytest.mark.parametrize("f32", [True, False])
def test_beam_select_equal_logits(tqlib, f32):
    """Rows of one value: equal scores of equal logits go by place, also where they are more than the list takes."""
    from turboquant_kv_cache_gb300 import binding as tb
    x = torch.full((2, 3, 128256), 0.5, device="cuda", dtype=torch.float32 if f32 else torch.float16)
    out = tb.tq_beam_select(x, torch.tensor([[-1.0, -1.0, -1.0], [-2.0, -1.0, -1.0]], device="cuda"), n_out=64)
    assert out[2].tolist() == [list(range(64))] * 2 and out[1].tolist() == [[0] * 64, [4] * 64]
