"""The fast quantiser serves every head_dim with one kernel per block size and
bit width: calls of any order of head_dims succeed and give the same records."""
import pytest
import torch

from turboquant_kv_cache_gb300 import inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("block,bits", [(32, 2), (32, 3), (32, 4), (64, 2), (64, 3), (64, 4)])
def test_head_dims_in_any_order(tqlib, block, bits):
    from turboquant_kv_cache_gb300 import binding as tb
    x = {d: torch.from_numpy(inputs.gaussian((300, d), d)).cuda() for d in (64, 128, 256)}
    first = {}
    for d in (256, 64, 128, 256, 64, 256, 128):
        p = tb.tq_quantize_kv(tb.make_layout(d, block, bits), x[d])
        torch.cuda.synchronize()
        if d in first:
            assert torch.equal(p.codes, first[d].codes) and torch.equal(p.scales, first[d].scales)
        first[d] = p
