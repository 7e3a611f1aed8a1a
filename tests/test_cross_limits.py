"""Cross attention at the ends of its arguments' ranges."""
import numpy as np
import pytest
import torch

from tests.test_step_refusals import _cross

pq = pytest.importorskip("paged_quantized_kv_cache_b200")

MOST = (2 ** 31 - 1) // 16 - 8  # blocks of a sequence: its positions, rounded up to two KV tiles, fit 32 bits


@pytest.mark.parametrize("most", [1, 400])
def test_tables_too_wide_are_refused(most):
    for width in (MOST + 1, MOST + 8, 2 ** 28):
        assert _cross(maxblk=width, most=most) == pq.ERR_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="the arguments are addresses that no kernel may see")
def test_the_widest_table_is_taken():
    assert _cross(maxblk=MOST) == _cross(maxblk=MOST, most=400) == pq.ERR_CUDA  # past the checks: there is no device


@pytest.mark.gpu
def test_a_bound_of_query_tokens_without_end():
    """max_q_len = 2^31 - 1 bounds every sequence: no row is past it."""
    from tests import step_reference as ref
    from tests.test_gpu_cross import _build, _run
    case = (pq.BF16, torch.bfloat16, 64, 1, 1)
    g, o, bt, cu, q, lens = _build(case, [100], [300], seed=51)
    out, err = _run(g, q, cu, bt, lens, 0.1, max_q_len=2 ** 31 - 1)
    want, tol = ref.cross(o, q, cu, bt, lens, 0.1)
    assert err == 0 and (np.abs(out.double().cpu().numpy() - want) <= tol).all()
