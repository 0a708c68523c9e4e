"""tq_decode_attn_shared where the scores are not those of unit Gaussians:
weights far below a slice's largest, references that move in the middle of a
slice, large scores.

The bounds.  The kernel rounds q^, k^ (rotated, per element), v^ and p to fp16,
half a step each: 2^-11 of the value.  Then
  * a score scale * <q^, k^> is off by 2 * 2^-11 * scale * |q| |k| at most
    (Cauchy-Schwarz; a rotation keeps norms), and its weight by the factor
    exp of that;
  * p, which is also what the sum l is made of, changes its weight by 2^-11
    more, and by 2^-30 of the reference's weight below fp16's normal range
    (the reference's p is 2^5, fp16's smallest step 2^-24);
  * a weight's factor e^x moves the output by w (e^x - 1) (v - out);
  * v^ moves an output component by 2^-11 sum w |v| (norms: the rotation back
    mixes a block's components);
  * the output is rounded once, 2^-11.
The fp32 sums between them are below a hundredth of these (2^-24 each)."""
import math

import numpy as np
import pytest
import torch

from turboquant_kv_cache_gb300 import inputs

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -11


def _attend(q, k, v, scale):
    """Outputs of q [H, R, d] over k, v [H, T, d] in 64 bits, and how far the
    kernel's may be from them."""
    s = torch.einsum("hrd,htd->hrt", q, k) * scale
    w = s.softmax(-1)
    out = w @ v
    x = 2 * HALF * scale * q.norm(dim=-1)[..., None] * k.norm(dim=-1)[:, None] + HALF
    grow = w * torch.expm1(x)
    tol = grow @ v.abs() + grow.sum(-1, keepdim=True) * out.abs()          # sum of grow |v - out|, from above
    tol = tol * x.amax(-1, keepdim=True).exp()                             # the weights' sum, which divides
    small = k.shape[1] * 2.0 ** -30                                        # all that p's smallest steps leave out
    tol += small * (v.abs().amax(1, keepdim=True) + out.abs())
    tol += HALF * (w * v.norm(dim=-1)[:, None]).sum(-1, keepdim=True) + HALF * out.abs() + 2.0 ** -25
    return out, 1.01 * tol


def _layout(tb, d, bits, block):
    return tb.make_layout(d, block, bits)


def _records(tb, L, which, factor, seed):
    """A cache [1, H, T] whose record (h, t) is vector which[t] of head h of a
    few quantised ones, its norms times factor[t]."""
    H = 2 if which.dim() == 1 else which.shape[0]
    x = torch.from_numpy(inputs.gaussian((1, H, int(which.max()) + 1, L.head_dim), seed)).cuda()
    base = tb.tq_quantize_kv(L, x)
    return tb.PackedKV.of(L, base.codes[:, :, which].contiguous(),
                          (base.scales[:, :, which].float() * factor[:, None]).half().contiguous())


@pytest.mark.parametrize("d,kbits,vbits,block", [(64, 4, 4, 64), (128, 3, 3, 32), (256, 4, 3, 32)])
def test_many_weights_far_below_the_largest(tqlib, d, kbits, vbits, block):
    """One token and 131071 of 2^-25.6 of its weight each, in one slice: they
    are 0.26 % of the softmax together, twice the library's 2e-3 at values of
    two."""
    from turboquant_kv_cache_gb300 import binding as tb
    T, down = 131072, 25.6
    first = torch.arange(T, device="cuda") == 0
    zero = torch.zeros(T, dtype=torch.long, device="cuda")
    K = _records(tb, _layout(tb, d, kbits, block), zero, first.float(), 1)
    V = _records(tb, _layout(tb, d, vbits, block), zero, (~first).float() * 2, 2)
    k = tb.tq_dequantize_kv(K, torch.float32)[0, :, 0].double()
    v = tb.tq_dequantize_kv(V, torch.float32)[0, :, 1].double()
    q = k.half()
    scale = down * math.log(2) / (q.double() * k).sum(-1)[0].item()
    lead = lambda c, h: tb.PackedKV.of(c.layout, c.codes[:, h:h + 1].contiguous(), c.scales[:, h:h + 1].contiguous())  # noqa: E731
    K, V = lead(K, 0), lead(V, 0)
    out = tb.tq_decode_attn_shared(K, V, K, V, q[None, :1].contiguous(), prefix_ctx=0, ctx=T, softmax_scale=scale, n_split=1)
    rest = (T - 1) * 2.0 ** -down
    ref = rest / (1 + rest) * v[0]
    # the first score, 25.6 in powers of two: q^ and k^ move it by 2 * 2^-11 of
    # itself (all products are squares), 0.025, so the weights by 1.8 %; p =
    # 2^-20.6 has steps of 2^-24, half of one is 2^-4.4 = 4.7 % of it; v^,
    # the output and the products of the two errors: below 0.5 %
    err = (out[0, 0].double() - ref).abs()
    assert (err <= 0.07 * ref.abs() + 0.002 * rest * v[0].norm()).all(), (err.max().item(), ref.abs().max().item())


def _levels(T, slice_tokens):
    """Tokens by their place in a slice: the first ones at no score (0), from
    its second tile on at half (1), a single one near its end at the full score
    (2); so is the last token of all, in a tile that is not whole."""
    u = torch.arange(T, device="cuda") % slice_tokens
    lv = (u >= 200).long()
    lv[u == slice_tokens - 7] = 2
    lv[-1] = 2
    return lv


@pytest.mark.parametrize("d,kbits,vbits,block", [(64, 4, 4, 64), (64, 2, 3, 32), (128, 3, 3, 32), (128, 4, 2, 128),
                                                 (256, 4, 3, 32), (256, 1, 4, 256)])
@pytest.mark.parametrize("where,B,Hq,Hkv", [("own", 3, 16, 2), ("own", 2, 2, 2), ("prefix", 5, 64, 16), ("prefix", 20, 64, 16),
                                            ("prefix", 37, 48, 12)])
def test_references_that_move_inside_a_slice(tqlib, d, kbits, vbits, block, where, B, Hq, Hkv):
    """Scores that pass the reference by 2^13 in a slice's second tile and by
    2^13 again near its end, in some of a CTA's rows: what was summed before
    has to be scaled, and the tokens at 2^-13 of the later ones are so many
    that they count."""
    from turboquant_kv_cache_gb300 import binding as tb
    G = Hq // Hkv
    # a slice of the own tokens is all of them (n_split 1); the prefix's 31
    # tiles make slices of four over 8 x 16 (or more, over fewer heads) CTAs
    T = 2317 if where == "own" else 3900
    lv = _levels(T, T if where == "own" else 512)
    which = lv[None].expand(Hkv, T)[0]
    one = torch.zeros_like(which)
    half = torch.tensor([0.0, 0.5, 1.0], device="cuda")[lv]

    def cache(bits, pick, factor, seed, n):
        L = _layout(tb, d, bits, block)
        x = torch.from_numpy(inputs.gaussian((1, Hkv, 3, d), seed)).cuda()
        c = tb.tq_quantize_kv(L, x)
        codes, scales = c.codes[:, :, pick], (c.scales[:, :, pick].float() * factor[:, None]).half()
        return tb.PackedKV.of(L, codes.expand(n, -1, -1, -1).contiguous(), scales.expand(n, -1, -1, -1).contiguous())

    n = B if where == "own" else 1
    K, V = cache(kbits, one, half, 3, n), cache(vbits, which, torch.ones_like(half), 4, n)
    k = tb.tq_dequantize_kv(K, torch.float32)[0].double()
    v = tb.tq_dequantize_kv(V, torch.float32)[0].double()
    full = k[:, -1]                                            # the vector at full score, per head
    # a row's share of that score: up, half as far (one move only), none, down
    share = torch.tensor([1.0, 0.5, 0.0, -1.0, 0.75], device="cuda", dtype=torch.float64)
    unit = full / full.norm(dim=-1, keepdim=True)
    rows = share[(torch.arange(B * Hq, device="cuda") % 5)].view(B, Hkv, G, 1)
    q = (rows * unit[None, :, None]).half()
    scale = 26 * math.log(2) / full.norm(dim=-1).max().item()
    q4 = q.view(B, Hq, d).contiguous()
    if where == "own":
        out = tb.tq_decode_attn_shared(K, V, K, V, q4, prefix_ctx=0, ctx=T, n_split=1, softmax_scale=scale)
    else:
        out = tb.tq_decode_attn_shared(K, V, None, None, q4, prefix_ctx=T, softmax_scale=scale)
    ref, tol = _attend(q.double().transpose(0, 1).reshape(Hkv, B * G, d), k, v, scale)
    got = out.view(B, Hkv, G, d).transpose(0, 1).reshape(Hkv, B * G, d).double()
    err = (got - ref).abs()
    assert (err <= tol).all(), (err / tol).max().item()
    # the bound tells: the outputs are far larger than it
    assert tol.max().item() < 0.25 * ref.abs().max().item()


@pytest.mark.parametrize("d,bits,block", [(64, 4, 32), (128, 3, 32), (256, 4, 32)])
@pytest.mark.parametrize("scale", [0.25, 1.0])
def test_large_scores_within_the_operands_roundings(tqlib, d, bits, block, scale):
    """Gaussian keys and queries at scales far above 1 / sqrt(d), prefix and
    own tokens."""
    from turboquant_kv_cache_gb300 import binding as tb
    B, Hq, Hkv, P, S = 3, 8, 2, 700, 150
    L = _layout(tb, d, bits, block)
    mk = lambda lead, seed: tb.tq_quantize_kv(L, torch.from_numpy(inputs.gaussian(lead + (d,), seed)).cuda())  # noqa: E731
    Kp, Vp, K, V = mk((1, Hkv, P), 11), mk((1, Hkv, P), 12), mk((B, Hkv, S), 13), mk((B, Hkv, S), 14)
    q = torch.from_numpy(inputs.gaussian((B, Hq, d), 15)).cuda()
    out = tb.tq_decode_attn_shared(Kp, Vp, K, V, q, softmax_scale=scale)
    dec = lambda c: tb.tq_dequantize_kv(c, torch.float32).double()  # noqa: E731
    for b in range(B):
        k, v = (torch.cat([dec(p)[0], dec(o)[b]], 1) for p, o in ((Kp, K), (Vp, V)))
        ref, tol = _attend(q[b].double().view(Hkv, Hq // Hkv, d), k, v, scale)
        err = (out[b].double().view_as(ref) - ref).abs()
        assert (err <= tol).all(), (err / tol).max().item()
