"""The scratch in which cross attention ranks its sequences lies where TMA copies
land next: its stores and loads are ordered before them by a proxy fence of every
thread, ahead of the barrier that they all pass before the first copy is issued."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_quantized_kv_cache_b200", "csrc")


def test_the_ranking_is_fenced_from_the_copies():
    with open(os.path.join(CSRC, "cross.cuh")) as f:
        body = re.search(r"int nth_longest\(.*?\n}\n", f.read(), re.S).group(0)
    last_use = max(m.end() for m in re.finditer(r"scratch\[", body))
    fence, barrier = body.find("fence_smem_to_async();", last_use), body.rfind("__syncthreads();")
    assert last_use < fence < barrier < body.rfind("return")
    with open(os.path.join(CSRC, "tcgen05.cuh")) as f:
        assert re.search(r"void fence_smem_to_async\(\) \{\s*asm volatile\(\"fence.proxy.async.shared::cta;\"", f.read())
