"""Every device function of the headers that wrap instructions has a kernel that
calls it."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_quantized_kv_cache_b200", "csrc")


@pytest.mark.parametrize("header", ["tcgen05.cuh", "cluster.cuh", "attn_math.cuh", "rope.cuh"])
def test_no_function_is_left_over(header):
    sources = {f: open(f).read() for f in glob.glob(os.path.join(CSRC, "*.cu*"))}
    text = sources[os.path.join(CSRC, header)]
    names = re.findall(r"(?:__forceinline__|constexpr)[^(;{=]*?(\w+)\(", text)
    assert names
    unused = [n for n in names if sum(len(re.findall(r"\b%s\b *[<(]" % n, t)) for t in sources.values()) < 2]
    assert not unused
