"""The ring of KV tiles of cross attention's many-row kernel, on the CPU.

With one row tile the halves of a CTA take the KV tiles in turn, and a wait for
a tile sees only the parity of its stage's phase. The model lets copies land in
any order and the halves drift apart, and looks for a half that reads a stage
before its tile is there, or a tile refilled before it was read."""
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_quantized_kv_cache_b200",
                      "csrc", "cross.cu")


def kernel_stages():
    with open(SOURCE) as f:
        return int(re.search(r"kStages = (\d+);", f.read()).group(1))


def fault(stages, tiles, seed):
    """What goes wrong in one random schedule (None: nothing)."""
    rnd = random.Random(seed)
    full, empty = [0] * stages, [0] * stages  # completed phases
    holds, read = [None] * stages, [True] * stages
    landing, landed, produced, nxt, ready = [], set(), 0, [0, 1], [0, 0]
    for now in range(20000):
        for copy in [c for c in landing if c[0] <= now]:
            landing.remove(copy)
            full[copy[1]] += 1
            landed.add(copy[2])
        if produced < tiles:
            s, lap = produced % stages, produced // stages & 1
            if produced < stages or empty[s] & 1 != lap ^ 1:
                if not read[s]:
                    return "refilled before it was read"
                holds[s], read[s] = produced, False
                landing.append((now + rnd.choice((3, 4, 5, 40)), s, produced))
                produced += 1
        for w in (0, 1):
            t = nxt[w]
            if t < tiles and now >= ready[w] and full[t % stages] & 1 != t // stages & 1:
                if t not in landed or holds[t % stages] != t:
                    return "read before its tile was there"
                empty[t % stages] += 1
                read[t % stages] = True
                nxt[w], ready[w] = t + 2, now + rnd.randint(1, 6)
        if min(nxt) >= tiles:
            return "copies in flight at the end" if landing else None
    return "stuck"


@pytest.mark.parametrize("tiles", [1, 2, 3, 5, 9, 23, 60])
def test_kernel_ring(tiles):
    assert [fault(kernel_stages(), tiles, seed) for seed in range(100)] == [None] * 100


def test_odd_ring_is_found_out():
    assert any(fault(5, 23, seed) for seed in range(100))
