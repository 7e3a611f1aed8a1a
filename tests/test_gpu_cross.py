"""Attention to an encoder's cached states (every format) against 64-bit
attention over the oracle's dequantized states."""
import numpy as np
import pytest
import torch

import oracle
from tests import gpu_helpers as gh
from tests import step_reference as ref
from tests.helpers import random_tables, slots

pytestmark = pytest.mark.gpu

pq = pytest.importorskip("paged_quantized_kv_cache_b200")

CASES = [
    # kv_dtype, q dtype, D, Hq, Hkv
    (pq.BF16, torch.bfloat16, 128, 32, 8),
    (pq.FP16, torch.float16, 64, 8, 2),
    (pq.BF16, torch.bfloat16, 64, 4, 4),
    (pq.FP16, torch.float16, 128, 16, 1),
    (pq.FP8_E4M3, torch.bfloat16, 128, 32, 8),
    (pq.FP8_E5M2, torch.float16, 64, 16, 2),
    (pq.FP4_E2M1, torch.bfloat16, 128, 32, 8),
    (pq.FP4_E2M1, torch.float16, 64, 8, 4),
]
ID = lambda c: "kv%d-D%d-G%d" % (c[0], c[2], c[3] // c[4])  # noqa: E731


def _build(case, lens, qlens, seed, wide=0, extra=3, share=False):
    kv_dtype, qdt, D, Hq, Hkv = case
    rng = np.random.default_rng(seed)
    nb = sum(-(-L // 16) for L in lens) + extra
    bt = random_tables(rng, lens, nb, max_blocks=max(1, max(-(-L // 16) for L in lens)) + wide)
    g, o = gh.new_pair(kv_dtype, nb, Hkv, D)
    in_dt = qdt
    for b, L in enumerate(lens):
        if L == 0:
            continue
        k, v = rng.standard_normal((2, L, Hkv, D)).astype(np.float32)
        if kv_dtype == pq.FP4_E2M1:
            for h in range(Hkv):
                k[:, h, rng.choice(D, 2, replace=False)] *= 16
                v[:, h, rng.choice(D, 2, replace=False)] *= 16
        kt, vt = torch.from_numpy(k).to(in_dt), torch.from_numpy(v).to(in_dt)
        ge, oe = gh.write_both(g, o, kt, vt, slots(bt[b], 0, L))
        assert ge == oe == 0
    if share:
        bt[1] = bt[0]
        lens = [lens[0], lens[0]] + list(lens[2:])
    cu = np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)
    q = torch.from_numpy(rng.standard_normal((int(cu[-1]), Hq, D)).astype(np.float32)).to(qdt)
    return g, o, bt, cu, q, list(lens)


def _run(g, q, cu, bt, lens, scale, ranges=None, max_q_len=None, stream=None):
    out = torch.full_like(q.cuda(), float("nan"))
    e = gh.err_flag()
    most = int(max(np.diff(cu))) if max_q_len is None else max_q_len
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()  # noqa: E731
    args = (q.cuda(), i32(cu), max(1, most), g, i32(bt), i32(lens), scale, out, e)
    kw = dict(kv_ranges=None if ranges is None else i32(ranges))
    torch.cuda.synchronize()
    pq.paged_cross_attention(*args, stream=stream, **kw)
    torch.cuda.synchronize()
    return out, int(e.item())


def _check(g, o, q, cu, bt, lens, scale, ranges=None, bits=0, **kw):
    out, err = _run(g, q, cu, bt, lens, scale, ranges, **kw)
    assert err == bits
    want, tol = ref.cross(o, q, cu, bt, lens, scale, ranges)
    got = out.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), "%d of %d outside; first %s: %r, not %r (+- %r)" % (
        bad.sum(), bad.size, np.argwhere(bad)[0], got[bad][0], want[bad][0], tol[bad][0])
    return out


def _ranges(rng, cu, lens):
    """Ranges of every kind: whole, empty, reversed, past both ends, one position, pieces across tiles."""
    r = np.zeros((int(cu[-1]), 2), np.int64)
    for b, L in enumerate(lens):
        for t in range(cu[b], cu[b + 1]):
            a, z = sorted(rng.integers(0, max(1, L) + 1, 2))
            kind = rng.integers(0, 7)
            r[t] = [(0, L), (a, a), (z, a), (-5, z), (a, L + 1000), (a, a + 1), (a, z)][kind]
    return r


@pytest.mark.parametrize("case", CASES, ids=ID)
def test_ragged_batch(case):
    """More and fewer query tokens than states, one token, tiles that end inside a block, several tile pairs."""
    lens, qlens = [333, 16, 1, 700, 65], [70, 40, 3, 1, 200]
    g, o, bt, cu, q, lens = _build(case, lens, qlens, seed=100 + case[0] + case[2])
    _check(g, o, q, cu, bt, lens, 1 / np.sqrt(case[2]))


@pytest.mark.parametrize("case", CASES, ids=ID)
def test_ranges_per_token(case):
    lens, qlens = [400, 129, 64], [90, 33, 7]
    g, o, bt, cu, q, lens = _build(case, lens, qlens, seed=200 + case[0] + case[2])
    _check(g, o, q, cu, bt, lens, 1 / np.sqrt(case[2]), _ranges(np.random.default_rng(1), cu, lens))


@pytest.mark.parametrize("L", [1, 15, 16, 17, 63, 64, 65, 128, 1500])
@pytest.mark.parametrize("case", [CASES[0], CASES[1], CASES[4], CASES[6]], ids=ID)
def test_one_token(case, L):
    """A decode step: few rows, the states split over a cluster (a wide table allows more parts than tiles)."""
    lens = [L, max(1, L // 2)]
    g, o, bt, cu, q, lens = _build(case, lens, [1, 1], seed=300 + L, wide=40)
    out = _check(g, o, q, cu, bt, lens, 1 / np.sqrt(case[2]))
    again, _ = _run(g, q, cu, bt, lens, 1 / np.sqrt(case[2]))
    assert torch.equal(out, again)


@pytest.mark.parametrize("case", [CASES[0], CASES[4], CASES[6]], ids=ID)
def test_one_token_each_is_the_decode(case):
    lens = [300, 41, 1000]
    g, o, bt, cu, q, lens = _build(case, lens, [1, 1, 1], seed=400)
    out = _check(g, o, q, cu, bt, lens, 0.09)
    dec, err = gh.decode_gpu(g, q, bt, lens, 0.09)
    want, tol = ref.cross(o, q, cu, bt, lens, 0.09)
    assert err == 0 and (np.abs(out.double().cpu().numpy() - dec.double().cpu().numpy()) <= 2 * tol).all()


@pytest.mark.parametrize("splits", [1, 2, 4, 8])
@pytest.mark.parametrize("case", [CASES[0], CASES[3], CASES[4], CASES[6]], ids=ID)
def test_every_split_of_the_states(case, splits):
    """Batches whose grids leave room for 1, 2, 4 and 8 parts; ranges that leave some parts without tiles."""
    Hkv = case[4]
    batch = {8: 1, 4: 3, 2: 6, 1: 10}[splits] if Hkv == 8 else {8: 10, 4: 30, 2: 60, 1: 100}[splits]
    lens, qlens = [900 - 7 * i for i in range(batch)], [5] * batch
    g, o, bt, cu, q, lens = _build(case, lens, qlens, seed=500)
    _check(g, o, q, cu, bt, lens, 0.1)
    r = np.tile([[0, 64]], (int(cu[-1]), 1))
    r[::3] = [130, 131]
    r[1::7] = [5, 5]
    _check(g, o, q, cu, bt, lens, 0.1, r)


FEW = [
    # query tokens a sequence; batch (8 KV heads: the states in 16, 8, 4, 2 and 1 parts)
    ([1], "one of 16 parts"), ([2, 1], "8 parts"), ([4, 0, 3, 1], "4 parts"), ([1, 2] * 4, "2 parts"), ([2] * 20, "1 part"),
]


@pytest.mark.parametrize("qlens", [f[0] for f in FEW], ids=[f[1] for f in FEW])
@pytest.mark.parametrize("case", CASES, ids=ID)
def test_a_few_tokens(case, qlens):
    """Up to 16 query rows per KV head, whole states and ranges (some without a position, some parts without a block)."""
    G = case[3] // case[4]
    qlens = [min(n, 16 // G) for n in qlens]
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(1, 1200, len(qlens))]
    g, o, bt, cu, q, lens = _build(case, lens, qlens, seed=700 + len(qlens), wide=20)
    _check(g, o, q, cu, bt, lens, 1 / np.sqrt(case[2]))
    _check(g, o, q, cu, bt, lens, 1 / np.sqrt(case[2]), _ranges(rng, cu, lens))


@pytest.mark.parametrize("batch", [40, 96, 97, 130, 193])
def test_many_sequences_of_a_few_tokens(batch):
    """More clusters than fit the GPU at once, taken in the order of their lengths (equal and empty ones among
    them) while a thread can rank a sequence, in the batch's order beyond."""
    case = (pq.FP8_E4M3, torch.bfloat16, 64, 8, 8)
    rng = np.random.default_rng(batch)
    lens = [int(x) for x in rng.integers(0, 60, batch)]
    qlens = [int(x) for x in rng.integers(0, 4, batch)]
    g, o, bt, cu, q, lens = _build(case, lens, qlens, seed=900 + batch)
    _check(g, o, q, cu, bt, lens, 0.125)


def test_few_tokens_edges():
    for case in (CASES[0], CASES[5], CASES[6]):
        g, o, bt, cu, q, lens = _build(case, [100, 0, 40, 260, 17], [1, 2, 0, 2, 1], seed=607)
        out = _check(g, o, q, cu, bt, lens, 0.1)
        assert (out[1:3] == 0).all()
        for scale in (0.0, -0.4, 15.0):
            _check(g, o, q, cu, bt, lens, scale)
        bt[0, 1], bt[3, 4], bt[3, 16] = g.num_blocks, -1, 2 ** 31 - 1
        _check(g, o, q, cu, bt, lens, 0.1, bits=pq.DEVERR_BLOCK_ID)
        lens[0], lens[4] = -3, 16 * bt.shape[1] + 1
        out = _check(g, o, q, cu, bt, lens, 0.1, bits=pq.DEVERR_BLOCK_ID | pq.DEVERR_SEQ_LEN)
        assert (out[0] == 0).all() and (out[-1] == 0).all()
        lens[0], lens[4] = 100, 17
        out, err = _run(g, q, cu, bt, lens, 0.1, max_q_len=1)  # the second tokens are not computed
        assert err == pq.DEVERR_BLOCK_ID | pq.DEVERR_SEQ_LEN and torch.isnan(out[2]).all() and not torch.isnan(out[3]).any()


# 1500 positions in 16 parts: every copy is issued at the start and may land before the first wait; 12 sequences of
# 3000: with 16-bit states the copies are what a warp waits for, and its waits run out; quantized states may be there
# (in L2) before the warp is done with the blocks before them
@pytest.mark.parametrize("lens", [[1500], [3000] * 12], ids=["short", "long"])
@pytest.mark.parametrize("case", [CASES[0], CASES[4], CASES[6]], ids=ID)
def test_few_tokens_wait_limit_runs_out_and_the_next_call_is_correct(case, lens):
    g, o, bt, cu, q, lens = _build(case, lens, [1] * len(lens), seed=608)
    seen = 0
    pq.set_decode_wait_limit_ns(1)
    try:
        for _ in range(5):
            _, e = _run(g, q, cu, bt, lens, 0.088)
            assert e & ~pq.DEVERR_TIMEOUT == 0
            seen += (e & pq.DEVERR_TIMEOUT) != 0
            if seen:
                break
    finally:
        pq.set_decode_wait_limit_ns(0)
    assert seen or len(lens) == 1 or case[0] != pq.BF16
    _check(g, o, q, cu, bt, lens, 0.088)


def _sloped(case, L, tokens, shape, seed):
    """Scores that run from -`top` to `top` (times a little noise) over the positions in the given shape: the row
    max moves at every tile, by much, at one position only, or never again after the first."""
    kv_dtype, qdt, D, Hq, Hkv = case
    rng = np.random.default_rng(seed)
    nb = -(-L // 16) + 1
    bt = random_tables(rng, [L], nb)
    g, o = gh.new_pair(kv_dtype, nb, Hkv, D)
    at = np.linspace(-1, 1, L)
    ramp = {"up": at, "down": -at, "spike": np.where(np.arange(L) == L - 40, 1, -0.2), "steps": np.floor(at * 3) / 3}[shape]
    k = (ramp[:, None, None] + 0.02 * rng.standard_normal((L, Hkv, D))).astype(np.float32)
    v = rng.standard_normal((L, Hkv, D)).astype(np.float32)
    assert gh.write_both(g, o, torch.from_numpy(k).to(qdt), torch.from_numpy(v).to(qdt), slots(bt[0], 0, L)) == (0, 0)
    q = torch.from_numpy((1 + 0.02 * rng.standard_normal((tokens, Hq, D))).astype(np.float32)).to(qdt)
    return g, o, q, np.array([0, tokens], np.int32), bt


@pytest.mark.parametrize("shape", ["up", "down", "spike", "steps"])
@pytest.mark.parametrize("top", [6, 60, 400])
@pytest.mark.parametrize("case", [CASES[0], CASES[1], CASES[4], CASES[6]], ids=ID)
def test_row_maxima_that_move(case, top, shape):
    """Exponents past what the standing max allows (2^15 for P in f16, 2^60 in bf16), in both kernels."""
    D = case[2]
    for tokens in (1, 70):
        g, o, q, cu, bt = _sloped(case, 700, tokens, shape, seed=800 + tokens)
        _check(g, o, q, cu, bt, [700], top / D)
        r = np.tile([[100, 650]], (tokens, 1))
        r[::3] = [0, 130]
        _check(g, o, q, cu, bt, [700], top / D, r)


@pytest.mark.parametrize("batch,Hkv", [(40, 8), (700, 1)])
def test_many_sequences_of_many_rows(batch, Hkv):
    """More CTAs than fit the GPU at once, in the order of the sequences' lengths, and past the number of
    sequences that the threads of a CTA can rank."""
    for kv_dtype, dtype in ((pq.BF16, torch.bfloat16), (pq.FP8_E5M2, torch.float16)):
        case = (kv_dtype, dtype, 64, 8 * Hkv, Hkv)
        rng = np.random.default_rng(batch)
        lens = [int(x) for x in rng.integers(0, 90, batch)]
        qlens = [int(x) for x in rng.integers(0, 4, batch)]
        qlens[3] = 3
        g, o, bt, cu, q, lens = _build(case, lens, qlens, seed=901 + batch)
        _check(g, o, q, cu, bt, lens, 0.125)


@pytest.mark.parametrize("tokens", [2, 24, 70])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("case", [CASES[0], CASES[1], CASES[3]], ids=ID)
def test_keys_that_a_token_does_not_see_may_hold_anything(case, value, tokens):
    kv_dtype, qdt, D, Hq, Hkv = case
    g, o, bt, cu, q, lens = _build(case, [640], [tokens], seed=17)
    ranges = np.array([[0, 320] if t % 2 else [320, 640] for t in range(tokens)], np.int32)
    want, tol = ref.cross(o, q, cu, bt, lens, 0.1, ranges)
    keys = g.cache.view(qdt).view(g.num_blocks, Hkv, 2, 16, D)
    for p in (0, 17, 319):  # positions that tokens of the second range do not see
        keys[int(bt[0, p // 16]), :, 0, p % 16] = value
    out, err = _run(g, q, cu, bt, lens, 0.1, ranges)
    assert err == 0
    assert (np.abs(out.double().cpu().numpy() - want) <= tol)[::2].all()


@pytest.mark.parametrize("scale", [0.0, -0.3, 8.0])
@pytest.mark.parametrize("case", [CASES[0], CASES[4]], ids=ID)
def test_other_scales_of_many_rows(case, scale):
    g, o, bt, cu, q, lens = _build(case, [200, 500], [30, 70], seed=605)
    _check(g, o, q, cu, bt, lens, scale)


def test_empty_and_rejected_sequences():
    case = CASES[1]
    lens, qlens = [40, 0, 30, 0, 20], [5, 4, 0, 1, 3]
    g, o, bt, cu, q, lens = _build(case, lens, qlens, seed=600)
    out = _check(g, o, q, cu, bt, lens, 0.125)
    assert (out[5:9] == 0).all() and (out[9] == 0).all()
    lens[0], lens[4] = 16 * bt.shape[1] + 1, -1
    out = _check(g, o, q, cu, bt, lens, 0.125, bits=pq.DEVERR_SEQ_LEN)
    assert (out[:5] == 0).all() and (out[10:] == 0).all()


def test_bad_block_ids_are_skipped():
    for case in (CASES[0], CASES[5], CASES[6]):
        g, o, bt, cu, q, lens = _build(case, [100, 260], [3, 150], seed=601)
        bt[0, 1], bt[1, 4], bt[1, 16] = g.num_blocks, -1, 2 ** 31 - 1
        _check(g, o, q, cu, bt, lens, 0.1, bits=pq.DEVERR_BLOCK_ID)


def test_rows_past_max_q_len_are_flagged_and_rows_behind_the_last_sequence_kept():
    case = CASES[1]
    g, o, bt, cu, q, lens = _build(case, [100, 70], [40, 2], seed=602)
    out, err = _run(g, q, cu, bt, lens, 0.125, max_q_len=16)
    assert err == pq.DEVERR_SEQ_LEN
    want, tol = ref.cross(o, q, cu, bt, lens, 0.125)
    got = out.double().cpu().numpy()
    assert (np.abs(got - want)[:32] <= tol[:32]).all() and (np.abs(got - want)[40:] <= tol[40:]).all()
    cu2 = np.array([0, 30, 35], np.int32)
    out, err = _run(g, q, cu2, bt, lens, 0.125)
    assert err == 0 and torch.isnan(out[35:]).all() and not torch.isnan(out[:35]).any()


def test_states_shared_by_two_sequences_and_moved_blocks_give_the_same_bits():
    case = CASES[4]
    g, o, bt, cu, q, lens = _build(case, [300, 300, 50], [4, 4, 60], seed=603, extra=24, share=True)
    q[cu[1]:cu[2]] = q[cu[0]:cu[1]]
    out = _check(g, o, q, cu, bt, lens, 0.09)
    assert torch.equal(out[cu[0]:cu[1]], out[cu[1]:cu[2]])
    used = set(int(x) for x in bt.ravel() if x >= 0)
    free = [i for i in range(g.num_blocks) if i not in used][:19]
    pairs = np.stack([bt[0, :19], free], axis=1).astype(np.int32)
    pq.copy_blocks(g, torch.from_numpy(pairs).cuda(), gh.err_flag())
    bt2 = bt.copy()
    bt2[0, :19] = free
    again, _ = _run(g, q, cu, bt2, lens, 0.09)
    assert torch.equal(out, again)


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3, 20.0])
def test_other_scales(scale):
    case = CASES[2]
    g, o, bt, cu, q, lens = _build(case, [200], [9], seed=604)
    _check(g, o, q, cu, bt, lens, scale)


def test_captured_replayed_and_on_another_stream():
    case = CASES[0]
    g, o, bt, cu, q, lens = _build(case, [500, 90], [1, 1], seed=605)
    out = _check(g, o, q, cu, bt, lens, 0.088, stream=torch.cuda.Stream())
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()  # noqa: E731
    gq, dst, e = q.cuda(), torch.empty_like(out), gh.err_flag()
    args = (gq, i32(cu), 1, g, i32(bt), i32(lens), 0.088, dst, e)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph in graphs:
        with torch.cuda.graph(graph):
            pq.paged_cross_attention(*args)
    for graph in graphs:
        dst.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dst, out)
    gq.copy_(gq.flip(0))
    graphs[0].replay()
    torch.cuda.synchronize()
    want, tol = ref.cross(o, gq.cpu(), cu, bt, lens, 0.088)
    assert (np.abs(dst.double().cpu().numpy() - want) <= tol).all() and int(e.item()) == 0


@pytest.mark.parametrize("case", [CASES[0], CASES[4], CASES[6]], ids=ID)
def test_wait_limit_runs_out_and_the_next_call_is_correct(case):
    """As the prefill's test of its timeout path, with split states: only the limit is short, nothing is dropped."""
    g, o, bt, cu, q, lens = _build(case, [1500], [40], seed=606)
    seen = 0
    pq.set_decode_wait_limit_ns(1)
    try:
        for _ in range(5):
            _, e = _run(g, q, cu, bt, lens, 0.088)
            assert e & ~pq.DEVERR_TIMEOUT == 0
            seen += (e & pq.DEVERR_TIMEOUT) != 0
            if seen:
                break
    finally:
        pq.set_decode_wait_limit_ns(0)
    assert seen
    _check(g, o, q, cu, bt, lens, 0.088)


@pytest.mark.parametrize("case", [CASES[0], CASES[1], CASES[4], CASES[6]], ids=ID)
def test_the_halves_of_a_row_tile_give_the_same_bits_from_cold_memory(case):
    # one row tile, whose halves take the KV tiles in turn, while the copies' latencies differ
    G = case[3] // case[4]
    lens = [1450 - 7 * b for b in range(16)]
    qlens = [32 // G] * 16
    g, o, bt, cu, q, lens = _build(case, lens, qlens, seed=91)
    _check(g, o, q, cu, bt, lens, 0.1)
    first = _run(g, q, cu, bt, lens, 0.1)[0]
    sweep = torch.empty(64 << 20, dtype=torch.int32, device="cuda")
    for i in range(12):
        sweep.fill_(i)
        out, err = _run(g, q, cu, bt, lens, 0.1)
        assert err == 0 and torch.equal(out.view(torch.int16), first.view(torch.int16))
