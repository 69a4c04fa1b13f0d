"""The debug build's promise for the sampling, rotary and page kernels: each store
to an output, a cache, the book-keeping or the workspace stands behind a check of its
place (``dcheck``).  CPU only: the sources are read; the GPU suite under
FP8RL_DEBUG=1 runs the checks themselves."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_w8a8_rollout_gb300", "csrc")

# stores through a pointer into an output or the workspace, by file
STORES = {
    "sample.cuh": r"\ba\.(tokens|lp|lp_kept|kept)\[r\] =",
    "rotary.cu": r"\*reinterpret_cast<uint[24]\*>\((to|code) \+|\b(to|code)\[c[01]\] =",
    "pages.cu": r"\ba\.(list|refs|lens|slots|to)\[[^\]]*\] =|\brow\[[^\]]*\] =|a\.row\[r\] =|a\.out\[.*\] =|a\.lens_out\[r\] =|"
                r"a\.copies\[[hm]\]\.(dst|src) =|\*at = a\.to|dst\[place\(",
}
NEAR = 20  # lines


@pytest.mark.parametrize("name", STORES)
def test_stores_stand_behind_checks(name):
    with open(os.path.join(CSRC, name)) as f:
        lines = [re.sub(r"//.*", "", line) for line in f]
    found = 0
    for i, line in enumerate(lines):
        if not re.search(STORES[name], line):
            continue
        found += 1
        above = lines[max(0, i - NEAR):i + 1]
        assert any("dcheck(" in a for a in above), (name, i + 1, line)
    assert found >= 4
