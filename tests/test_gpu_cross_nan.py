"""Cross attention where a score that a token sees is not a number: the token's
row is NaN in every channel, whatever the split of the states and the shape of
the launch, and no other row is touched by it."""
import numpy as np
import pytest
import torch

from tests import step_reference as ref
from tests.test_gpu_cross import CASES, ID, _build, _run

pytestmark = pytest.mark.gpu

pq = pytest.importorskip("paged_quantized_kv_cache_b200")

# with 8 KV heads: sequences, query rows per KV head of each. Up to 16 rows: the few-rows kernel; up to 128: one row
# tile, whose halves share the KV tiles; above: two row tiles. Few sequences: the states in several parts
SHAPES = {"few, parts": (1, 8), "few": (20, 8), "one tile, parts": (1, 40), "one tile": (20, 40), "two tiles, parts": (1, 200),
          "two tiles": (20, 200)}
L = 300
PLACES = [70, 299]  # the second and the last KV tile, which the halves of a row tile take
QUARTER = [CASES[0], CASES[1], CASES[4], CASES[6]]


def _state(case, shape):
    """Sequences as `shape` says, of L states each, and the one to spoil."""
    G = case[3] // case[4]
    batch, rows = SHAPES[shape]
    batch = max(1, batch * 8 // case[4]) if batch > 1 else 1
    tokens = rows // G
    g, o, bt, cu, q, lens = _build(case, [L] * batch, [tokens] * batch, seed=rows + batch, wide=60)
    return g, o, bt, cu, q, lens, batch // 2


def _check_rows(out, want, tol, bad):
    """`bad` [T][Hq]: rows that are NaN throughout; all others are right."""
    got = out.double().cpu().numpy()
    nan = np.isnan(got)
    assert (nan.all(-1) == bad).all() and (nan.any(-1) == bad).all(), "%d rows are NaN, not %d" % (nan.any(-1).sum(), bad.sum())
    assert (np.abs(got - want) <= tol)[~bad].all()


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("case", QUARTER, ids=ID)
def test_a_query_of_nan_gives_a_row_of_nan(case, shape):
    g, o, bt, cu, q, lens, b = _state(case, shape)
    want, tol = ref.cross(o, q, cu, bt, lens, 0.1)
    bad = np.zeros(q.shape[:2], bool)
    for t, h, what in ((cu[b], 0, slice(None)), (cu[b + 1] - 1, case[3] - 1, 5), (cu[b + 1] - 1, 1, case[2] - 1)):
        q[t, h, what] = float("nan")
        bad[t, h] = True
    out, err = _run(g, q, cu, bt, lens, 0.1)
    assert err == 0
    _check_rows(out, want, tol, bad)


@pytest.mark.parametrize("place", PLACES)
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("case", QUARTER[:3], ids=ID)
def test_a_key_of_nan_gives_nan_where_it_is_seen(case, shape, place):
    kv_dtype, qdt, D, Hq, Hkv = case
    g, o, bt, cu, q, lens, b = _state(case, shape)
    G = Hq // Hkv
    ranges = np.tile([[0, L]], (q.shape[0], 1))
    ranges[1::2] = [place + 1, L] if place < L // 2 else [0, place]
    want, tol = ref.cross(o, q, cu, bt, lens, 0.1, ranges)
    h, block = Hkv - 1, int(bt[b, place // 16])
    if kv_dtype == pq.FP8_E4M3:
        g.cache.view(-1, Hkv, 2, 16, D)[block, h, 0, place % 16, 7] = 0x7F
    else:
        g.cache.view(qdt).view(-1, Hkv, 2, 16, D)[block, h, 0, place % 16, 7] = float("nan")
    bad = np.zeros(q.shape[:2], bool)
    bad[cu[b]:cu[b + 1], h * G:] = (ranges[cu[b]:cu[b + 1], 0] <= place)[:, None] & (ranges[cu[b]:cu[b + 1], 1] > place)[:, None]
    out, err = _run(g, q, cu, bt, lens, 0.1, ranges)
    assert err == 0
    _check_rows(out, want, tol, bad)
    # and without ranges every token of the sequence sees it
    want, tol = ref.cross(o, q, cu, bt, lens, 0.1)
    bad[cu[b]:cu[b + 1], h * G:] = True
    out, err = _run(g, q, cu, bt, lens, 0.1)
    assert err == 0
    _check_rows(out, want, tol, bad)
