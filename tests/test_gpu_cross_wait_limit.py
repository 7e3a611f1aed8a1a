"""Cross attention whose waits give up: a row is left as it was, or it is right.
Only the limit is short; nothing is dropped, and the call after is correct."""
import numpy as np
import pytest
import torch

from tests import step_reference as ref
from tests.test_gpu_cross import CASES, ID, _build, _run

pytestmark = pytest.mark.gpu

pq = pytest.importorskip("paged_quantized_kv_cache_b200")

# (sequences, query rows per KV head): the states of a row in several parts, or in one; the halves of a CTA
SHAPES = {"few, parts": (3, 4), "few": (40, 4), "one tile, parts": (2, 40), "one tile": (40, 40), "two tiles, parts": (2, 200)}


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("case", [CASES[0], CASES[4], CASES[6]], ids=ID)
def test_rows_are_right_or_untouched(case, shape):
    batch, rows = SHAPES[shape]
    tokens = rows // (case[3] // case[4])
    long = 3000 if batch < 40 else 700
    g, o, bt, cu, q, lens = _build(case, [long + 16 * b for b in range(batch)], [tokens] * batch, seed=608)
    want, tol = ref.cross(o, q, cu, bt, lens, 0.088)
    sweep = torch.empty(64 << 20, dtype=torch.int32, device="cuda")
    for limit in (1, 1, 1500, 3000):
        sweep.fill_(limit)  # cold states: the copies take longer
        pq.set_decode_wait_limit_ns(limit)
        try:
            out, err = _run(g, q, cu, bt, lens, 0.088)
        finally:
            pq.set_decode_wait_limit_ns(0)
        assert err & ~pq.DEVERR_TIMEOUT == 0
        got = out.double().cpu().numpy()
        kept, right = np.isnan(got).all(-1), (np.abs(got - want) <= tol).all(-1)
        assert (kept | right).all(), "%d of %d rows are neither" % ((~(kept | right)).sum(), right.size)
        assert err or right.all()
    out, err = _run(g, q, cu, bt, lens, 0.088)
    assert err == 0 and (np.abs(out.double().cpu().numpy() - want) <= tol).all()
