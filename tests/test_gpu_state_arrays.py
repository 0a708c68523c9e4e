"""What a StateArrays refuses after it was made, and sizes that its C structs do not hold."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_cache_that_became_paged_is_refused(tqlib):
    """A paged cache's first dimension is its pages, not its sequences: the call
    refuses it also where the cache was contiguous when the StateArrays was made."""
    from turboquant_kv_cache_gb300 import binding as tb
    cache = tb.tq_quantize_kv(tb.make_layout(64, 32, 4), torch.randn(4, 2, 32, 64, device="cuda").half())
    states, parent = tb.StateArrays([cache]), i32([1, 0, 3, 2])
    codes = cache.codes.clone()
    tb.tq_states_reorder(states, parent, 4)
    assert torch.equal(cache.codes, codes[[1, 0, 3, 2]])
    codes = cache.codes.clone()
    cache.page_table = i32([[0, 1], [2, 3]])
    with pytest.raises(ValueError):
        tb.tq_states_reorder(states, parent, 4)
    assert torch.equal(cache.codes, codes)
    cache.page_table = None
    tb.tq_states_reorder(states, parent, 4)
    assert torch.equal(cache.codes, codes[[1, 0, 3, 2]])


@pytest.mark.parametrize("shape", [(1, 1, 1, 2**32 + 16), (1, 2**32 + 1, 1)])
def test_sizes_past_32_bits_are_refused(tqlib, shape):
    """Slots of 4 GB and more, or as many heads: a slot of 2^32 + 16 bytes is not one of 16."""
    from turboquant_kv_cache_gb300 import binding as tb
    with pytest.raises(ValueError):
        tb.StateArrays([torch.empty(shape, dtype=torch.uint8, device="cuda")])
