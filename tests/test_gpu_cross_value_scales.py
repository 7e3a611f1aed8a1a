"""FP8 states whose values differ by many powers of two between blocks: a token's
row is as exact as the blocks that it sees, and that carry weight, allow."""
import numpy as np
import pytest
import torch

from tests import gpu_helpers as gh
from tests import step_reference as ref
from tests.helpers import random_tables, slots
from tests.test_gpu_cross import _run

pytestmark = pytest.mark.gpu

pq = pytest.importorskip("paged_quantized_kv_cache_b200")

CASES = [(pq.FP8_E4M3, torch.bfloat16, 128, 32, 8), (pq.FP8_E5M2, torch.float16, 64, 8, 2),
         (pq.FP8_E4M3, torch.float16, 128, 16, 4), (pq.FP8_E5M2, torch.bfloat16, 64, 16, 2)]
ID = lambda c: "kv%d-D%d-G%d" % (c[0], c[2], c[3] // c[4])  # noqa: E731
HALF = 336  # states of each picture: 21 blocks, so that a KV tile holds blocks of both


def _build(case, tokens, sizes, seed, bias=None):
    """Pictures of HALF states whose values have standard deviation sizes[i], and whose keys, with `bias`, give every
    token scores that are about bias[i] larger (scale 1, log e units)."""
    kv_dtype, dtype, D, Hq, Hkv = case
    rng = np.random.default_rng(seed)
    L = HALF * len(sizes)
    bt = random_tables(rng, [L], L // 16 + 2)
    g, o = gh.new_pair(kv_dtype, L // 16 + 2, Hkv, D)
    k, v = rng.standard_normal((2, L, Hkv, D)).astype(np.float32)
    q = rng.standard_normal((tokens, Hq, D)).astype(np.float32)
    k *= 0.1
    if bias is not None:
        q[..., 0] = 1
        k[..., 0] = np.repeat(bias, HALF)[:, None]
    v *= np.repeat(np.array(sizes, np.float32), HALF)[:, None, None]
    assert gh.write_both(g, o, torch.from_numpy(k).to(dtype), torch.from_numpy(v).to(dtype), slots(bt[0], 0, L)) == (0, 0)
    for ours, theirs in zip(g.arrays(), o.arrays()):  # the attention is tested here, not the write of such values
        if ours is not None:
            theirs[:] = ours.cpu().numpy()
    return g, o, bt, torch.from_numpy(q).to(dtype), L


# fp16 inputs hold values of 2^-12 of one another only
RATIOS = {torch.bfloat16: [2.0 ** -12, 2.0 ** -20, 2.0 ** -28, 2.0 ** -60], torch.float16: [2.0 ** -8, 2.0 ** -12]}


@pytest.mark.parametrize("tokens", [2, 24, 70])
@pytest.mark.parametrize("case,ratio", [(c, r) for c in CASES for r in RATIOS[c[1]]],
                         ids=lambda x: ID(x) if isinstance(x, tuple) else "2^%.0f" % np.log2(x))
def test_values_that_a_token_does_not_see_do_not_change_its_row(case, ratio, tokens):
    """Each token sees one of two pictures: its row against 64-bit attention to that picture alone, whose tolerance
    knows nothing of the other's values."""
    for order in ((1.0, ratio), (ratio, 1.0)):
        g, o, bt, q, L = _build(case, tokens, order, seed=31)
        ranges = np.array([[0, HALF] if t % 2 else [HALF, L] for t in range(tokens)])
        cu = np.array([0, tokens], np.int32)
        out, err = _run(g, q, cu, bt, [L], 0.3, ranges)
        assert err == 0
        got = out.double().cpu().numpy()
        for first in (True, False):
            mine = np.arange(tokens) % 2 == int(first)
            table = bt[:, :HALF // 16] if first else bt[:, HALF // 16:]
            want, tol = ref.cross(o, q[mine], np.array([0, mine.sum()]), table, [HALF], 0.3, max_q_len=tokens)
            assert (np.abs(got[mine] - want) <= tol).all()


@pytest.mark.parametrize("tokens", [2, 24, 70])
@pytest.mark.parametrize("order", ["small first", "large first", "small last of three"])
def test_large_values_of_no_weight_leave_the_others_exact(tokens, order):
    """A token sees a picture of tiny values, at high scores, and one of values 2^40 times as large whose weights are
    below 2^-57. P enters its product with V in f16, in units of the largest p s so far (s: the V scale of a key's
    block, c = v / s its code): half a step of p s 2^-11, or 2^-25 units below 2^-14 of one, in either case times |c|.
    The unit is at most the largest p s of what the row sees, U."""
    case = CASES[0]
    sizes, bias = {"small first": ((2.0 ** -40, 1.0), (20.0, -20.0)), "large first": ((1.0, 2.0 ** -40), (-20.0, 20.0)),
                   "small last of three": ((1.0, 2.0 ** -20, 2.0 ** -40), (-20.0, 0.0, 20.0))}[order]
    g, o, bt, q, L = _build(case, tokens, sizes, seed=32, bias=np.array(bias, np.float32))
    cu = np.array([0, tokens], np.int32)
    want, wide = ref.cross(o, q, cu, bt, [L], 1.0)
    out, err = _run(g, q, cu, bt, [L], 1.0)
    assert err == 0
    import oracle
    kv_dtype, dtype, D, Hq, Hkv = case
    G = Hq // Hkv
    tol = np.empty_like(want)
    for h in range(Hkv):
        k, v, ok = oracle.gather(o, bt[0], L, h)
        s_v = np.repeat(o.scales.view(np.float32).reshape(-1, Hkv, 4)[bt[0, :L // 16], h, 1].astype(np.float64), 16)
        for n in range(h * G, (h + 1) * G):
            x = q[:, n].double().numpy() @ k.T
            size = np.abs(q[:, n].double().numpy()) @ np.abs(k).T
            p = np.exp(x - x.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            unit = (p * s_v).max(-1, keepdims=True)
            shift = (D * 2.0 ** -24 * size + 4 * 2.0 ** -24 * (np.abs(x) * 1.4427 + 8)).max(-1, keepdims=True)
            rel = 2.0 ** -11 + 2 * shift + 2 * L * 2.0 ** -24 + 2.0 ** -22
            tol[:, n] = ref.HALF[dtype] * np.abs(want[:, n]) + (1 + ref.HALF[dtype]) * (
                rel * (p @ np.abs(v)) + 2.0 ** -24 * unit * np.abs(v / s_v[:, None]).sum(0)) + ref.TINY[dtype]
    assert tol.max() < 2.0 ** -20 * wide.max()  # the other tolerance would pass zeros
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("tokens", [2, 70])
@pytest.mark.parametrize("size", [2.0 ** -115, 2.0 ** -120, 2.0 ** -122], ids=lambda s: "2^%.0f" % np.log2(s))
def test_values_near_the_smallest_normal_number(size, tokens):
    """V scales around 2^-126 and below, down to where their reciprocal is no float. The unit of P is at least
    2^-126, so that half its smallest subnormal may come to 2^-25 2^-126 times a code a key."""
    for case in (CASES[0], CASES[3]):
        for sizes in ((size, size), (0.0, size), (size, 0.0)):
            g, o, bt, q, L = _build(case, tokens, sizes, seed=33)
            cu = np.array([0, tokens], np.int32)
            want, tol = ref.cross(o, q, cu, bt, [L], 0.3)
            tol = tol + 2.0 ** -151 * L * (448 if case[0] == pq.FP8_E4M3 else 57344)
            assert size < 2.0 ** -120 or tol.max() < 2.0 ** -4 * size
            out, err = _run(g, q, cu, bt, [L], 0.3)
            assert err == 0 and (np.abs(out.double().cpu().numpy() - want) <= tol).all()
