"""Cross attention over bf16 values near 2^69 while the scores rise by 58 powers of
two from the first KV tile to the next ones: sums stay inside the range of fp32."""
import numpy as np
import pytest
import torch

from tests import gpu_helpers as gh
from tests import step_reference as ref
from tests.helpers import random_tables, slots
from tests.test_gpu_cross import _run

pytestmark = pytest.mark.gpu

pq = pytest.importorskip("paged_quantized_kv_cache_b200")


@pytest.mark.parametrize("tokens", [2, 20, 70])
@pytest.mark.parametrize("L", [128, 400])
def test_scores_that_rise_over_large_values(L, tokens):
    D, Hq, Hkv = 64, 8, 2
    rng = np.random.default_rng(41)
    bt = random_tables(rng, [L], L // 16)
    g, o = gh.new_pair(pq.BF16, L // 16, Hkv, D)
    k = 0.02 * rng.standard_normal((L, Hkv, D)).astype(np.float32)
    k[:, :, 0] = np.where(np.arange(L) < 64, 0, 53 * np.log(2))[:, None]
    v = (2.0 ** 69 * rng.uniform(0.5, 1, (L, Hkv, D))).astype(np.float32)
    q = 0.02 * rng.standard_normal((tokens, Hq, D)).astype(np.float32)
    q[..., 0] = 1
    kt, vt, qt = (torch.from_numpy(x).to(torch.bfloat16) for x in (k, v, q))
    assert gh.write_both(g, o, kt, vt, slots(bt[0], 0, L)) == (0, 0)
    cu = np.array([0, tokens], np.int32)
    want, tol = ref.cross(o, qt, cu, bt, [L], 1.0)
    out, err = _run(g, qt, cu, bt, [L], 1.0)
    assert err == 0 and (np.abs(out.double().cpu().numpy() - want) <= tol).all()
