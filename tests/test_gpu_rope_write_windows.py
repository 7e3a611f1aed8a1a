"""The fused quantized write of more than 8192 tokens, whose warps walk windows of
32 tokens: the bits of the two calls that it stands for, and of calls of fewer
tokens each."""
import numpy as np
import pytest
import torch

from tests import gpu_helpers as gh
from tests.test_gpu_rope import _cuda, _make, _views

pytestmark = pytest.mark.gpu

pq = pytest.importorskip("paged_quantized_kv_cache_b200")

CASES = [
    # kv_dtype, dtype, D, Hq, Hkv, interleaved
    (pq.FP8_E4M3, torch.bfloat16, 128, 4, 2, False),
    (pq.FP8_E5M2, torch.float16, 64, 2, 1, True),
    (pq.FP4_E2M1, torch.bfloat16, 128, 2, 1, True),
    (pq.FP4_E2M1, torch.float16, 64, 4, 2, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "kv%d-D%d-%s" % (c[0], c[2], "il" if c[5] else "half"))
def test_windows_of_tokens_give_the_bits_of_the_two_calls(case):
    kv_dtype, dtype, D, Hq, Hkv, il = case
    before, T, nb = 5, 8309, 545
    a, b, c = (pq.allocate_cache(kv_dtype, nb, Hkv, D, fill=gh.POISON) for _ in range(3))
    ids = np.random.default_rng(2).permutation(nb)
    for begin, n in ((0, before), (before, T)):
        x, w, pos, ax, table = _make(n, Hq, Hkv, D, dtype, D // 2, 2, seed=60 + n)
        p = begin + np.arange(n)
        slots = (ids[p // 16] * 16 + p % 16).astype(np.int32)
        if n == T:  # a request of its own after 4000 tokens: a block not filled; a skipped stretch; a bad position
            slots[4000:] = ids[270 + (np.arange(n - 4000)) // 16] * 16 + np.arange(n - 4000) % 16
            slots[1003:1051] = -1
            pos[1, 2000] = -3
        s, gp = torch.from_numpy(slots).cuda(), torch.from_numpy(pos).cuda()
        q, k, v = _views(x.cuda(), Hq, Hkv, D)
        rotary, kw = pq.Rotary(table.cuda(), ax, il), dict(q_weight=_cuda(w[0]), k_weight=_cuda(w[1]))
        qa, qb, qc = (torch.full((n, Hq, D), float("nan"), dtype=dtype, device="cuda") for _ in range(3))
        ka, errs = torch.empty(n, Hkv, D, dtype=dtype, device="cuda"), [gh.err_flag() for _ in range(3)]
        pq.qkv_norm_rope_write(q, k, v, gp, rotary, qa, s, a, errs[0], **kw)
        pq.qk_norm_rope(q, k, gp, rotary, qb, ka, errs[1], **kw)
        pq.kv_cache_write(ka, v.contiguous(), s, b, errs[1])
        cuts = [0, n] if n == before else [0, 11, 1003, 3995, 4000, 4000 + 16 * 200, n]  # where blocks begin
        for i, j in zip(cuts, cuts[1:]):
            pq.qkv_norm_rope_write(q[i:j], k[i:j], v[i:j], gp[:, i:j].contiguous(), rotary, qc[i:j], s[i:j].contiguous(), c, errs[2], **kw)
        torch.cuda.synchronize()
        assert [int(e.item()) for e in errs] == [pq.DEVERR_POSITION if n == T else 0] * 3
        bits = lambda t: t.contiguous().view(torch.int16)  # noqa: E731
        assert torch.equal(bits(qa), bits(qb)) and torch.equal(bits(qa), bits(qc))
        for one, two, three in zip(a.arrays(), b.arrays(), c.arrays()):
            if one is not None:
                assert torch.equal(one, two) and torch.equal(one, three)
