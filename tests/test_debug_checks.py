"""The debug build's promise for the norm, attention and log-probability kernels:
each store to an output or a workspace stands behind a check of its place
(``dcheck``).  CPU only: the sources are read; the GPU suite under FP8RL_DEBUG=1
runs the checks themselves."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_w8a8_rollout_gb300", "csrc")

# stores through a pointer into an output or the workspace, by file
STORES = {
    "norm.cu": r"\*reinterpret_cast<uint[24]\*>\((row|qr) \+|\b(hr|qr)\[[^\]]*\] =|\(a\.scale\)\[[^\]]*\] =",
    "attn_decode.cu": r"\*reinterpret_cast<\w+\*>\((to|a\.out) \+|\b(a\.out|a\.lse|to)\[.*?\] =|atomicAdd\(ticket|\*ticket =",
    "attn_prefill.cu": r"st_global_v8\(|\*reinterpret_cast<uint4\*>\(to( \+ 8)?\) =|\ba\.lse\[[^\]]*\] =",
    "logprob.cu": r"__stcs\(|\bstore1<In>\(|\ba\.(lp|entropy|stats|top_ids|top_lp)\[[^\]]*\] =",
}
NEAR = 45  # lines


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
