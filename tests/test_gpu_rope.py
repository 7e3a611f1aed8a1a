"""Norm and rotation of query and key heads, alone and with the cache write,
against 64-bit arithmetic and against the calls they stand for."""
import numpy as np
import pytest
import torch

from tests import gpu_helpers as gh
from tests import step_reference as ref

pytestmark = pytest.mark.gpu

pq = pytest.importorskip("paged_quantized_kv_cache_b200")

DT = {torch.float16: pq.FP16, torch.bfloat16: pq.BF16}


def _table(count, rot, seed=0):
    f = 10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))
    a = np.arange(count)[:, None] * f
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1)).float()


def _make(T, Hq, Hkv, D, dtype, rot, axes, seed, norm=True, count=5000, gap=0):
    """A projection's output with `gap` unused elements behind a token's heads; views of it, and the rest."""
    rng = np.random.default_rng(seed)
    width = (Hq + 2 * Hkv) * D
    size = np.exp(rng.uniform(-2, 2, width))
    x = torch.zeros(T, width + gap, dtype=dtype)
    x[:, :width] = torch.from_numpy(rng.standard_normal((T, width)) * size).to(dtype)
    w = [torch.from_numpy(1 + 0.3 * rng.standard_normal(D)).float() if norm else None for _ in range(2)]
    pos = rng.integers(0, count, (axes, T)).astype(np.int32)
    ax = bytes(rng.integers(0, axes, rot // 2).astype(np.uint8).tolist()) if axes > 1 else b""
    return x, w, pos, ax, _table(count, rot)


def _views(x, Hq, Hkv, D):
    T = x.shape[0]
    return [x[:, a * D:b * D].view(T, b - a, D) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv))]


def _cuda(w):
    return None if w is None else w.cuda()


def _close(out, x, weight, eps, pos, ax, table, il):
    z, size = ref.norm_rope(x, weight, eps, pos, ax, table, il)
    got = out.double().cpu().numpy()
    bad = ~(np.abs(got - z) <= ref.rope_tolerance(z, size, x.dtype))
    assert not bad.any(), "%d of %d outside; first %s: %r, not %r" % (
        bad.sum(), bad.size, np.argwhere(bad)[0], got[bad][0], z[bad][0])


CASES = [
    # T, Hq, Hkv, D, rot, axes, interleaved, norm
    (1, 32, 8, 128, 128, 3, False, True),
    (1, 1, 1, 64, 64, 1, True, True),
    (3, 5, 3, 64, 32, 2, False, True),
    (37, 8, 2, 64, 56, 4, True, True),
    (130, 32, 8, 128, 64, 2, True, True),
    (67, 7, 1, 128, 8, 1, False, True),
    (29, 9, 3, 128, 120, 3, False, False),
    (50, 8, 4, 64, 0, 1, False, True),
    (18, 3, 2, 128, 128, 4, True, False),
    (1031, 16, 2, 64, 64, 1, False, True),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c))
def test_norm_rope_matches_64_bits(case, dtype):
    T, Hq, Hkv, D, rot, axes, il, norm = case
    x, w, pos, ax, table = _make(T, Hq, Hkv, D, dtype, rot, axes, seed=T + Hq, norm=norm, gap=8 * (T % 3))
    gx = x.cuda()
    q, k, _ = _views(gx, Hq, Hkv, D)
    qo, ko = (torch.full((T, h, D), float("nan"), dtype=dtype, device="cuda") for h in (Hq, Hkv))
    err = gh.err_flag()
    pq.qk_norm_rope(q, k, torch.from_numpy(pos).cuda(), pq.Rotary(table.cuda(), ax, il), qo, ko, err,
                    q_weight=_cuda(w[0]), k_weight=_cuda(w[1]), eps=1e-5)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.equal(gx.cpu(), x)
    hq, hk, _ = _views(x, Hq, Hkv, D)
    _close(qo, hq, w[0], 1e-5, pos, ax, table if rot else None, il)
    _close(ko, hk, w[1], 1e-5, pos, ax, table if rot else None, il)


def test_in_place_alone_and_without_keys():
    x, w, pos, ax, table = _make(77, 8, 2, 64, torch.bfloat16, 64, 1, seed=3)
    q, k, _ = (v.cuda().contiguous() for v in _views(x, 8, 2, 64))
    p, rotary, err = torch.from_numpy(pos[0]).cuda(), pq.Rotary(table.cuda()), gh.err_flag()
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    pq.qk_norm_rope(q, k, p, rotary, qo, ko, err, q_weight=w[0].cuda())
    only = torch.empty_like(q)
    pq.qk_norm_rope(q, None, p, rotary, only, None, err, q_weight=w[0].cuda())
    pq.qk_norm_rope(q, k, p, rotary, q, k, err, q_weight=w[0].cuda())
    plain = torch.empty_like(k)
    pq.qk_norm_rope(ko, None, None, None, plain, None, err)  # nothing to do: a copy
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(only, qo) and torch.equal(plain, ko)


def test_rows_of_zeros_and_of_extremes():
    """A row of zeros stays zero for any eps above 0; rows near the ends of the types' ranges keep their norm."""
    for dtype, big, small in ((torch.bfloat16, 1e15, 1e-15), (torch.float16, 60000.0, 1e-4)):
        x, w, pos, ax, table = _make(4, 3, 1, 128, dtype, 128, 1, seed=4)
        x = (x.float() / x.float().abs().max()).to(dtype)
        x[0] = 0
        x[1] = (x[1].float() * big).to(dtype)
        x[2] = (x[2].float() * small).to(dtype)
        q, k, _ = _views(x.cuda(), 3, 1, 128)
        qo, ko, err = torch.empty(4, 3, 128, dtype=dtype, device="cuda"), torch.empty(4, 1, 128, dtype=dtype, device="cuda"), gh.err_flag()
        pq.qk_norm_rope(q, k, torch.from_numpy(pos).cuda(), pq.Rotary(table.cuda()), qo, ko, err, q_weight=w[0].cuda(),
                        k_weight=w[1].cuda(), eps=1e-12)
        assert (qo[0] == 0).all()
        hq, hk, _ = _views(x, 3, 1, 128)
        _close(qo, hq, w[0], 1e-12, pos, ax, table, False)
        _close(ko, hk, w[1], 1e-12, pos, ax, table, False)


def test_a_position_outside_the_table_zeros_the_token():
    x, w, pos, ax, table = _make(40, 8, 2, 64, torch.float16, 64, 2, seed=5)
    pos[0, 3], pos[1, 17], pos[1, 30] = -1, 5000, 2 ** 31 - 1
    q, k, _ = _views(x.cuda(), 8, 2, 64)
    qo, ko, err = torch.empty_like(q, memory_format=torch.contiguous_format), torch.empty(40, 2, 64, dtype=x.dtype, device="cuda"), gh.err_flag()
    qo = torch.empty(40, 8, 64, dtype=x.dtype, device="cuda")
    pq.qk_norm_rope(q, k, torch.from_numpy(pos).cuda(), pq.Rotary(table.cuda(), ax), qo, ko, err, q_weight=w[0].cuda())
    torch.cuda.synchronize()
    assert int(err.item()) == pq.DEVERR_POSITION
    for t in (3, 17, 30):
        assert (qo[t] == 0).all() and (ko[t] == 0).all()
    hq, hk, _ = _views(x, 8, 2, 64)
    _close(qo, hq, w[0], 1e-6, pos, ax, table, False)
    _close(ko, hk, None, 1e-6, pos, ax, table, False)


WRITE = [
    # kv_dtype, dtype, D, Hq, Hkv, interleaved
    (pq.BF16, torch.bfloat16, 128, 32, 8, False),
    (pq.FP16, torch.float16, 64, 8, 2, True),
    (pq.FP8_E4M3, torch.bfloat16, 128, 32, 8, False),
    (pq.FP8_E4M3, torch.float16, 64, 8, 4, True),
    (pq.FP8_E5M2, torch.bfloat16, 64, 8, 2, False),
    (pq.FP8_E5M2, torch.float16, 128, 4, 1, True),
    (pq.FP4_E2M1, torch.bfloat16, 128, 32, 8, False),
    (pq.FP4_E2M1, torch.float16, 128, 8, 2, True),
    (pq.FP4_E2M1, torch.bfloat16, 64, 8, 8, False),
]


@pytest.mark.parametrize("case", WRITE, ids=lambda c: "kv%d-D%d-%s" % (c[0], c[2], "il" if c[5] else "half"))
def test_the_write_in_one_call_is_the_two_calls(case):
    """Chunks that open, fill and append to blocks, a skipped token, and one slot too far: the cache's bytes,
    the queries and the error bits of the two calls it stands for."""
    kv_dtype, dtype, D, Hq, Hkv, il = case
    nb, rot = 12, D // 2
    a, b = (pq.allocate_cache(kv_dtype, nb, Hkv, D, fill=gh.POISON) for _ in range(2))
    ids = np.random.default_rng(1).permutation(nb)
    begin = 0
    for step, n in enumerate((37, 1, 1, 60, 5)):
        x, w, pos, ax, table = _make(n, Hq, Hkv, D, dtype, rot, 3, seed=10 + step, norm=step != 3)
        p = begin + np.arange(n)
        slots = ids[p // 16] * 16 + p % 16
        if step == 3:
            slots[40] = -1
        if step == 4:
            slots[4] = nb * 16
        begin += n
        gx = x.cuda()
        q, k, v = _views(gx, Hq, Hkv, D)
        s, gp = torch.from_numpy(slots.astype(np.int32)).cuda(), torch.from_numpy(pos).cuda()
        rotary, ea, eb = pq.Rotary(table.cuda(), ax, il), gh.err_flag(), gh.err_flag()
        qa, qb = (torch.full((n, Hq, D), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
        kb = torch.empty(n, Hkv, D, dtype=dtype, device="cuda")
        pq.qk_norm_rope(q, k, gp, rotary, qb, kb, eb, q_weight=_cuda(w[0]), k_weight=_cuda(w[1]))
        pq.kv_cache_write(kb, v.contiguous(), s, b, eb)
        pq.qkv_norm_rope_write(q, k, v, gp, rotary, qa, s, a, ea, q_weight=_cuda(w[0]), k_weight=_cuda(w[1]))
        torch.cuda.synchronize()
        assert int(ea.item()) == int(eb.item()) == (pq.DEVERR_SLOT if step == 4 else 0)
        assert torch.equal(qa, qb)
        for x1, x2 in zip(a.arrays(), b.arrays()):
            assert (x1 is None) == (x2 is None)
            if x1 is not None:
                assert torch.equal(x1, x2), "step %d" % step


def test_a_bad_position_writes_a_zero_key():
    x, w, pos, ax, table = _make(20, 4, 2, 64, torch.bfloat16, 64, 1, seed=40)
    pos[0, 5] = 5000
    q, k, v = _views(x.cuda(), 4, 2, 64)
    slots = torch.arange(16, 36, dtype=torch.int32, device="cuda")
    for kv_dtype in (pq.BF16, pq.FP8_E4M3):
        c, err = pq.allocate_cache(kv_dtype, 3, 2, 64, fill=0), gh.err_flag()
        qo = torch.empty(20, 4, 64, dtype=x.dtype, device="cuda")
        pq.qkv_norm_rope_write(q, k, v, torch.from_numpy(pos).cuda(), pq.Rotary(table.cuda()), qo, slots, c, err,
                               k_weight=w[1].cuda())
        torch.cuda.synchronize()
        assert int(err.item()) == pq.DEVERR_POSITION and (qo[5] == 0).all()
        rows = c.cache.view(3, 2, 2, 16, -1)[1, :, :, 5]
        assert (rows[:, 0] & 0x7F == 0).all() and (rows[:, 1] != 0).any()


def test_captured_and_on_another_stream():
    x, w, pos, ax, table = _make(50, 8, 2, 64, torch.bfloat16, 64, 1, seed=50)
    gx, p, rotary, err = x.cuda(), torch.from_numpy(pos).cuda(), pq.Rotary(table.cuda()), gh.err_flag()
    c = pq.allocate_cache(pq.FP8_E4M3, 8, 2, 64, fill=0)
    slots = torch.arange(50, dtype=torch.int32, device="cuda")
    qo = torch.empty(50, 8, 64, dtype=x.dtype, device="cuda")
    wk = w[1].cuda()

    def call(stream=None):
        pq.qkv_norm_rope_write(*_views(gx, 8, 2, 64), p, rotary, qo, slots, c, err, k_weight=wk, stream=stream)

    torch.cuda.synchronize()
    call(stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    want, cache = qo.clone(), c.cache.clone()
    gx.mul_(2)  # the queries are not normed here: they double; the normed keys' codes stay
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(qo, want * 2)
    k_rows = lambda t: t.view(8, 2, 2, 16, 64)[:3, :, 0]  # noqa: E731
    assert (k_rows(c.cache) == k_rows(cache)).float().mean() > 0.9
    assert int(err.item()) == 0


# T, Hq, Hkv, D, interleaved: enough rows that a warp takes two, and four, groups of them; head counts that end inside a group
GROUPS = [(330, 250, 9, 128, False), (650, 250, 9, 128, True), (650, 245, 33, 128, False), (1400, 250, 17, 64, True),
          (340, 250, 50, 64, False)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("case", GROUPS, ids=lambda c: "-".join(str(x) for x in c))
def test_many_rows_give_the_bits_of_few(case, dtype):
    """One call of many tokens, in place too, and calls of 20 tokens each; a bad position among them; with the write."""
    T, Hq, Hkv, D, il = case
    rot, axes = D - 8, 3
    x, w, pos, ax, table = _make(T, Hq, Hkv, D, dtype, rot, axes, seed=31)
    pos[1, T // 2] = -7
    gx, gp, rotary = x.cuda(), torch.from_numpy(pos).cuda(), pq.Rotary(table.cuda(), ax, il)
    q, k, v = _views(gx, Hq, Hkv, D)
    kw = dict(q_weight=w[0].cuda(), k_weight=w[1].cuda())
    new = lambda n, h: torch.full((n, h, D), float("nan"), dtype=dtype, device="cuda")  # noqa: E731
    qa, ka, err = new(T, Hq), new(T, Hkv), gh.err_flag()
    pq.qk_norm_rope(q, k, gp, rotary, qa, ka, err, **kw)
    qi, ki = q.contiguous(), k.contiguous()
    pq.qk_norm_rope(qi, ki, gp, rotary, qi, ki, err, **kw)
    qb, kb = new(T, Hq), new(T, Hkv)
    for t in range(0, T, 20):
        n = slice(t, min(T, t + 20))
        pq.qk_norm_rope(q[n], k[n], gp[:, n].contiguous(), rotary, qb[n], kb[n], err, **kw)
    cache = pq.allocate_cache(DT[dtype], -(-T // 16), Hkv, D, fill=gh.POISON)
    qc, slots = new(T, Hq), torch.randperm(T, generator=torch.Generator().manual_seed(1)).int().cuda()
    pq.qkv_norm_rope_write(q, k, v, gp, rotary, qc, slots, cache, err, **kw)
    torch.cuda.synchronize()
    assert int(err.item()) == pq.DEVERR_POSITION
    bits = lambda t: t.contiguous().view(torch.int16)  # noqa: E731
    for got, want in ((qa, qb), (ka, kb), (qi, qb), (ki, kb), (qc, qb)):
        assert torch.equal(bits(got), bits(want))
    rows = cache.cache.view(dtype).view(-1, Hkv, 2, 16, D).permute(0, 3, 1, 2, 4).reshape(-1, Hkv, 2, D)[slots.long()]
    assert torch.equal(bits(rows[:, :, 0]), bits(kb)) and torch.equal(bits(rows[:, :, 1]), bits(v))
    pick = [0, 1, T // 2, T - 1]
    _close(qa[pick], _views(x, Hq, Hkv, D)[0][pick], w[0], 1e-6, pos[:, pick], ax, table, il)
    _close(ka[pick], _views(x, Hq, Hkv, D)[1][pick], w[1], 1e-6, pos[:, pick], ax, table, il)


@pytest.mark.parametrize("case", GROUPS[:2], ids=lambda c: "-".join(str(x) for x in c))
def test_many_rows_without_norm_and_rotation_are_copied(case):
    T, Hq, Hkv, D, il = case
    x = _make(T, Hq, Hkv, D, torch.bfloat16, 0, 1, seed=32)[0].cuda()
    q, k, _ = _views(x, Hq, Hkv, D)
    qo, ko = (torch.empty(T, h, D, dtype=x.dtype, device="cuda") for h in (Hq, Hkv))
    pq.qk_norm_rope(q, k, None, None, qo, ko, gh.err_flag())
    torch.cuda.synchronize()
    assert torch.equal(qo, q) and torch.equal(ko, k)
