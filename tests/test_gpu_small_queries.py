"""bf16 queries of quantized caches whose largest value is below 2^-114, down to
the smallest subnormal: the scores are next to nothing, so that a row is about
the mean of the values it sees, in every attention over the cache."""
import numpy as np
import pytest
import torch

import oracle
from tests import gpu_helpers as gh
from tests import step_reference as ref
from tests.test_gpu_cross import CASES, ID, _build, _run

pytestmark = pytest.mark.gpu

pq = pytest.importorskip("paged_quantized_kv_cache_b200")

SIZES = [2.0 ** -110, 1e-36, 2.0 ** -126, 2.0 ** -130, 2.0 ** -133]
BF16_Q = [c for c in CASES if c[1] == torch.bfloat16 and c[0] not in (pq.BF16, pq.FP16)] + [(pq.FP8_E5M2, torch.bfloat16, 64, 16, 2)]


def _shrink(q, size):
    """Rows of this size, among them one channel alone (zeros beside it) and a row of zeros."""
    q = (q.double() * size).to(q.dtype)
    q[0, 0] = 0
    q[0, 0, 3] = size
    q[0, 1] = 0
    return q


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "2^%.0f" % np.log2(s))
@pytest.mark.parametrize("tokens", [2, 50])
@pytest.mark.parametrize("case", BF16_Q, ids=ID)
def test_cross_attention(case, tokens, size):
    g, o, bt, cu, q, lens = _build(case, [300, 41], [tokens, 1], seed=11)
    q = _shrink(q, size)
    want, tol = ref.cross(o, q, cu, bt, lens, 0.1)
    out, err = _run(g, q, cu, bt, lens, 0.1)
    assert err == 0 and (np.abs(out.double().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "2^%.0f" % np.log2(s))
@pytest.mark.parametrize("case", BF16_Q, ids=ID)
def test_decode_and_prefill(case, size):
    kv_dtype, dtype, D, Hq, Hkv = case
    lens = [300, 41]
    g, o, bt, cu, q, lens = _build(case, lens, [1, 1], seed=12)
    q = _shrink(q, size)
    out, err = gh.decode_gpu(g, q, bt, lens, 0.1)
    want, rerr = oracle.paged_decode(o, q, bt, lens, 0.1)
    assert err == rerr == 0
    gh.assert_close(out, want, kv_dtype, tag="decode")
    cu = np.array([0, 200, 241], np.int32)
    q = _shrink(torch.randn(241, Hq, D, generator=torch.Generator().manual_seed(1)).to(dtype), size)
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()  # noqa: E731
    out, e = torch.empty_like(q.cuda()), gh.err_flag()
    pq.paged_prefill_attention(q.cuda(), i32(cu), 200, g, i32(bt), i32(lens), 0.1, out, e)
    torch.cuda.synchronize()
    want, rerr = oracle.paged_prefill(o, q, cu, bt, lens, 0.1)
    assert int(e.item()) == rerr == 0
    gh.assert_close(out, want, kv_dtype, tag="prefill")
