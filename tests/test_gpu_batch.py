"""The batch's tables built on the GPU, against the plain implementation: every
output equal, the rest of the block tables as it was."""
import numpy as np
import pytest
import torch

from tests import step_reference as ref

pytestmark = pytest.mark.gpu

pq = pytest.importorskip("paged_quantized_kv_cache_b200")


def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(x, np.int32)).cuda()


def _case(rng, B, past, new_hi, extra_cols=2):
    start = rng.integers(0, past + 1, B)
    new = rng.integers(0, new_hi + 1, B)
    have, need = -(-start // 16), -(-(start + new) // 16)
    most = max(1, int(need.max())) + extra_cols
    nb = int(need.sum()) + 9
    pool = rng.permutation(nb)
    fresh = int((need - have).sum())
    tables = np.full((B, most), -7, np.int64)
    tables[np.arange(most)[None] < have[:, None]] = pool[fresh:fresh + int(have.sum())]
    return start, new, pool[:fresh], tables, nb


def _run(start, new, ids, tables, nb, capacity, stream=None):
    t, e = _i32(tables), torch.zeros(1, dtype=torch.int32, device="cuda")
    B = len(start)
    out = [torch.full((n,), -99, dtype=torch.int32, device="cuda") for n in (capacity, capacity, B + 1, B)]
    pq.build_batch(_i32(start), _i32(new), _i32(ids), t, nb, *out, e, stream=stream)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in (t, *out)] + [int(e.item())]


def _check(args, capacity):
    got, want = _run(*args, capacity), ref.batch(*args, capacity)
    for name, g, w in zip(("tables", "slots", "positions", "cu", "lens"), got, want):
        np.testing.assert_array_equal(g, w, err_msg=name)
    assert got[5] == want[5]
    return want


@pytest.mark.parametrize("B", [1, 2, 31, 255, 256, 257, 1000, pq.MAX_BATCH])
@pytest.mark.parametrize("past,new_hi", [(0, 40), (200, 1), (100, 33)])
def test_batch_matches_the_plain_form(B, past, new_hi):
    rng = np.random.default_rng(B * 7 + past + new_hi)
    args = _case(rng, B, past, new_hi)
    T = int(args[1].sum())
    _check(args, T)
    _check(args, T + 301)


def test_no_new_tokens_anywhere():
    args = _case(np.random.default_rng(5), 7, 60, 0)
    _check(args, 0)
    _check(args, 12)


def test_no_requests():
    _check((np.zeros(0, int), np.zeros(0, int), np.zeros(0, int), np.zeros((0, 4), int), 5), 9)


def test_bad_lengths_leave_a_request_empty():
    args = _case(np.random.default_rng(6), 9, 50, 20)
    start, new, ids, tables, nb = args
    most = tables.shape[1]
    for b, s, n in ((1, -1, 4), (3, 2, -5), (5, 16 * most, 1), (7, 2 ** 31 - 1, 2 ** 31 - 1)):
        start[b], new[b] = s, n
    want = _check((start, new, ids, tables, nb), 400)
    assert want[5] & ref.ERR_SEQ_LEN and list(want[4][[1, 3, 5, 7]]) == [0] * 4


@pytest.mark.parametrize("short", ["tokens", "blocks"])
def test_requests_that_do_not_fit_are_left_out_whole(short):
    args = _case(np.random.default_rng(8), 40, 30, 40)
    start, new, ids, tables, nb = args
    T = int(new.sum())
    want = _check(args, T - 1 - int(new[30:].sum())) if short == "tokens" else _check((start, new, ids[:20], tables, nb), T)
    assert want[5] == ref.ERR_CAPACITY and want[4][-1] == 0


def test_bad_block_ids():
    start, new, ids, tables, nb = _case(np.random.default_rng(9), 12, 40, 40)
    ids[2], ids[5] = nb, -3
    b = int(np.flatnonzero((start % 16 != 0) & (new > 0))[0])
    tables[b, start[b] // 16] = nb + 4  # the block that the request's next token goes into
    want = _check((start, new, ids, tables, nb), int(new.sum()))
    assert want[5] == ref.ERR_BLOCK_ID and (want[1] == -1).any()


def test_a_captured_call_follows_its_lengths():
    """One graph, replayed with other lengths and ids in the same buffers."""
    rng = np.random.default_rng(10)
    B, most, nb, cap = 20, 12, 400, 600
    start, new, ids = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (B, B, 200))
    tables = torch.zeros(B, most, dtype=torch.int32, device="cuda")
    out = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in (cap, cap, B + 1, B)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pq.build_batch(start, new, ids, tables, nb, *out, err)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pq.build_batch(start, new, ids, tables, nb, *out, err)
    for _ in range(3):
        s, n = rng.integers(0, 100, B), rng.integers(0, 30, B)
        i, t = rng.permutation(nb)[:200], rng.integers(0, nb, (B, most))
        for dst, src in ((start, s), (new, n), (ids, i), (tables, t)):
            dst.copy_(_i32(src))
        graph.replay()
        torch.cuda.synchronize()
        want = ref.batch(s, n, i, t, nb, cap)
        for g, w in zip((tables, *out), want):
            np.testing.assert_array_equal(g.cpu().numpy(), w)
        assert int(err.item()) == want[5] == 0


def test_another_stream():
    args = _case(np.random.default_rng(11), 33, 90, 25)
    stream = torch.cuda.Stream()
    T = int(args[1].sum())
    got, want = _run(*args, T, stream=stream), ref.batch(*args, T)
    for g, w in zip(got, want):
        np.testing.assert_array_equal(g, w)


@pytest.mark.parametrize("shift", [0, 1, 2, 3])
@pytest.mark.parametrize("left", [0, 1, 2, 3, 700])
def test_many_rows_in_arrays_of_any_alignment(shift, left):
    """Several rows a thread: results that start on any word, rows left over, empty requests, bad ids, padding."""
    rng = np.random.default_rng(40 + left)
    start, new, ids, tables, nb = _case(rng, 3000, 60, 70)
    new[rng.random(3000) < 0.3] = 0
    need = int((-(-(start + new) // 16) - -(-start // 16)).sum())
    ids = np.array(ids)[:need]
    ids[[0, need // 2, need - 1]] = nb, -1, nb + 7
    T = int(new.sum())
    cap = T + left
    room = [torch.full((cap + 8,), 77, dtype=torch.int32, device="cuda") for _ in range(2)]
    slots, positions = (r[shift:shift + cap] for r in room)
    t, cu, lens = _i32(tables).cuda(), torch.empty(3001, dtype=torch.int32, device="cuda"), torch.empty(3000, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pq.build_batch(_i32(start).cuda(), _i32(new).cuda(), _i32(ids).cuda(), t, nb, slots, positions, cu, lens, err)
    torch.cuda.synchronize()
    want = ref.batch(start, new, ids, tables, nb, cap)
    for got, w in zip((t, slots, positions, cu, lens), want):
        np.testing.assert_array_equal(got.cpu().numpy(), w)
    assert int(err.item()) == want[5] == ref.ERR_BLOCK_ID
    for r in room:
        assert (r[:shift] == 77).all() and (r[shift + cap:] == 77).all()
