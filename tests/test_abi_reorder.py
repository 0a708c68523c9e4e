"""tq_pages_reorder refuses arrays that are not aligned to their elements, on the host."""
import ctypes

import pytest

from turboquant_kv_cache_gb300 import binding as tb

ALIGN = -3


@pytest.mark.parametrize("which", ["parent", "seqs", "result"])
def test_pages_reorder_unaligned_arrays(tqlib, which):
    pool = tb.tq_page_pool(1 << 20, 1 << 20, 1 << 20, 16, 8, 64, 64)
    at = {"parent": 1 << 20, "seqs": 1 << 20, "result": 1 << 20}
    at[which] += 2
    st = tqlib.tq_pages_reorder(ctypes.byref(pool), at["parent"], at["seqs"], 8, at["result"], 1 << 20, 1 << 20, None)
    assert st == ALIGN
