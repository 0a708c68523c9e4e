"""Layouts that the tensor-core quantiser does not take (fp32 rows, rotation blocks
of 128 and 256, 1 bit): codes against the oracle, and byte for byte against the
kernel that compares with every boundary, which a layout with norm correction runs
on (it changes the norms alone).  Vectors whose rotated values lie on boundaries,
zeros, huge, tiny and non-finite ones among them."""
import numpy as np
import pytest
import torch

from oracle import tq_oracle as O
from turboquant_kv_cache_gb300 import inputs

from _parity import compare_codes, compare_scales, to_np

pytestmark = pytest.mark.gpu

F16, F32 = np.float16, np.float32
CASES = [  # d, block, bits, dtype
    *[(d, blk, bits, F32) for d, blk in ((64, 32), (64, 64), (128, 32), (128, 128), (256, 64), (256, 128), (256, 256))
      for bits in (1, 2, 3, 4)],
    *[(d, blk, bits, F16) for d, blk in ((128, 128), (256, 128), (256, 256)) for bits in (1, 2, 3, 4)],
    (64, 32, 1, F16), (64, 64, 1, F16), (128, 64, 1, F16), (256, 32, 1, F16),
]


def on_boundaries(n, L, seed):
    """Vectors whose rotated, normalised values are boundaries in three of four places."""
    rng = np.random.default_rng(seed)
    _, bnd = O.codebook_for(L)
    y = np.empty((n, L.d // L.blk, L.blk))
    for r in y.reshape(-1, L.blk):
        while True:
            v = rng.standard_normal(L.blk) / np.sqrt(L.blk)
            v = bnd[np.abs(v[:, None] - bnd).argmin(1)]
            free = rng.permutation(L.blk)[:L.blk // 4]
            v[free] = 0.0
            if v @ v < 1:
                break
        v[free] = rng.choice([-1.0, 1.0], len(free)) * np.sqrt((1 - v @ v) / len(free))
        r[:] = v
    h = O.hadamard_matrix(L.blk)
    x = (y @ h).reshape(n, L.d) * O.sign_vector(L.seed, L.d)
    return x * np.exp2(rng.integers(-3, 4, size=(n, 1)))


def rows_of(L, dt, seed):
    x = inputs.gaussian((701, L.d), seed, np.float32)
    x[3] = 0.0
    x[5] *= 300.0
    x[7] = 1.0
    x[9] = 0.0
    x[9, L.d - 1] = -2.0                        # every rotated value of a block +-1/sqrt(block)
    x[11, ::2] = 0.0
    x[13, 1::2] = -x[13, ::2]
    x[40, :32] = 0.0
    return np.concatenate([x, on_boundaries(300, L, seed)]).astype(dt)


@pytest.mark.parametrize("d,blk,bits,dt", CASES)
def test_codes_and_norms(tqlib, d, blk, bits, dt):
    from turboquant_kv_cache_gb300 import binding as tb
    L, Lo = tb.make_layout(d, blk, bits, sign_seed=1), O.Layout(d, blk, bits, 0, 0, 1)
    x = rows_of(Lo, dt, d + blk + bits)
    xg = torch.from_numpy(x).cuda()
    pk = tb.tq_quantize_kv(L, xg)
    oq = O.quantize(x, Lo)
    n_code, rows = compare_codes(to_np(pk.codes)[:701], {k: v[:701] for k, v in oq.items() if k in ("codes", "y")}, Lo)
    assert n_code <= 5 + 701 * d // 10000 + 3 * d   # rows 7, 9 and 13 have values that cancel: all of them may be ties
    compare_codes(to_np(pk.codes), oq, Lo)
    compare_scales(to_np(pk.scales), oq["scale"])
    assert np.all(to_np(pk.scales)[3] == 0)
    # the same codes as by comparison with each boundary, whatever the rows hold
    odd = x[:64].astype(np.float32)
    odd[0], odd[1, 5], odd[2, 7], odd[4, ::3], odd[6] = np.nan, np.nan, np.inf, -np.inf, np.inf
    if dt is F32:
        odd[8:16] *= 1e30
        odd[16:24] *= 1e-30
        odd[24:32] *= 1e-41
        odd[32:40] = np.finfo(np.float32).max
    else:
        odd[8:16] *= 1e-7
        odd[32:40] = 65504.0
    every = torch.cat([xg, torch.from_numpy(odd.astype(dt)).cuda()])
    got = tb.tq_quantize_kv(L, every)
    want = tb.tq_quantize_kv(tb.make_layout(d, blk, bits, norm_correct=1, sign_seed=1), every)
    assert torch.equal(got.codes, want.codes)


@pytest.mark.parametrize("d,blk,bits,dt", CASES[::3])
def test_rows_into_slots(tqlib, d, blk, bits, dt):
    """The same records behind the slots of a ragged batch."""
    from turboquant_kv_cache_gb300 import binding as tb
    L, Lo = tb.make_layout(d, blk, bits, sign_seed=1), O.Layout(d, blk, bits, 0, 0, 1)
    x = torch.from_numpy(rows_of(Lo, dt, d + bits)[:999]).cuda().view(333, 3, d)
    cache = tb.PackedKV(L, (12, 3, 32))
    cache.codes.fill_(0xA5)
    cache.scales.fill_(-1.0)
    slot = torch.randperm(12 * 32, device="cuda")[:333]
    slot[::7] = -1
    tb.tq_append_kv_slots(cache, x, slot)
    flat = tb.tq_quantize_kv(L, x)
    codes, scales = torch.full_like(cache.codes, 0xA5), torch.full_like(cache.scales, -1.0)
    live = slot >= 0
    codes[slot[live] // 32, :, slot[live] % 32] = flat.codes[live]
    scales[slot[live] // 32, :, slot[live] % 32] = flat.scales[live]
    assert torch.equal(cache.codes, codes) and torch.equal(cache.scales, scales)
