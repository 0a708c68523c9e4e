"""Where the kernels move registers between their warps.

`setmaxnreg.sync.aligned` is for whole warpgroups: all four warps execute the
same instruction.  So a role of fewer warps must not have an instruction of its
own; each direction stands once in a kernel, in front of the branches of the
roles that it is for."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "turboquant_kv_cache_gb300", "csrc")


def _branches(name):
    """The conditions under which each setmaxnreg of a file stands: the lines
    of the enclosing `if` / `else if` of one indentation less."""
    lines = open(os.path.join(CSRC, name)).read().split("\n")
    found = []
    for i, line in enumerate(lines):
        if "asm" not in line or "setmaxnreg" not in line:
            continue
        depth = len(line) - len(line.lstrip())
        for j in range(i - 1, -1, -1):
            up = lines[j]
            if up.strip() and not up.startswith("#") and len(up) - len(up.lstrip()) < depth:
                found.append((re.search(r"\.(inc|dec)\.", line).group(1), up.strip()))
                break
    return found


@pytest.mark.parametrize("name,whole", [
    # conditions that hold for whole warpgroups (4 warps) only
    ("tq_shared_tc.cu", [("dec", "if (warp >= kSoftWarps) {"), ("inc", "} else {")]),
    ("tq_prefill_tc.cu", [("dec", "if (warp >= 4) {"), ("inc", "} else {")]),
])
def test_one_register_split_per_warpgroup(name, whole):
    assert _branches(name) == whole
