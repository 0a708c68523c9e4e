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
