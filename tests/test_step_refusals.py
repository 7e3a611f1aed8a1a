"""Arguments that the operators around a serving step refuse, on the host and
before any launch, and the plain implementations that their GPU tests use."""
import ctypes

import numpy as np
import pytest
import torch

from tests import step_reference as ref

pq = pytest.importorskip("paged_quantized_kv_cache_b200")

F = ctypes.c_float
A = 1 << 20  # stands for an aligned device pointer: every call below is refused before it is used


def _batch(**kw):
    a = dict(start=A, new=2 * A, batch=4, ids=3 * A, n_ids=3, tables=4 * A, maxblk=8, nb=64, cap=10, slots=5 * A,
             pos=6 * A, cu=7 * A, lens=8 * A, err=9 * A)
    a.update(kw)
    return pq.lib().pqkv_build_batch(a["start"], a["new"], a["batch"], a["ids"], a["n_ids"], a["tables"], a["maxblk"],
                                     a["nb"], a["cap"], a["slots"], a["pos"], a["cu"], a["lens"], a["err"], None)


@pytest.mark.parametrize("bad", [
    dict(batch=-1), dict(batch=pq.MAX_BATCH + 1), dict(n_ids=-1), dict(maxblk=0), dict(maxblk=1 << 28), dict(nb=0),
    dict(nb=1 << 28), dict(cap=-1), dict(start=None), dict(new=None), dict(ids=None), dict(tables=None),
    dict(slots=None), dict(pos=None), dict(cu=None), dict(lens=None), dict(err=None),
    dict(lens=A), dict(cu=A - 16), dict(slots=2 * A + 12), dict(tables=3 * A - 124), dict(pos=5 * A + 36),
    dict(lens=7 * A + 16)], ids=str)
def test_batch_refuses(bad):
    assert _batch(**bad) == pq.ERR_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="the arguments are addresses that no kernel may see")
@pytest.mark.parametrize("good", [dict(), dict(cu=A - 20), dict(slots=2 * A + 16), dict(ids=None, n_ids=0), dict(new=A)],
                         ids=str)
def test_batch_takes_arrays_side_by_side(good):
    assert _batch(**good) == pq.ERR_CUDA  # past the checks: there is no device


def _rope(write=False, **kw):
    a = dict(q=A, k=2 * A, v=3 * A, dt=pq.BF16, T=4, hq=8, hkv=2, d=64, qs=512, ks=128, vs=128, qw=None, kw=None,
             eps=1e-6, pos=A, axes=1, axis=None, table=A, n=16, rot=64, il=0, q_out=4 * A, k_out=5 * A, err=A,
             slots=A, cache=6 * A, scales=A, oidx=A, oval=A, kv=pq.BF16, nb=64)
    a.update(kw)
    mid = [a["qw"], a["kw"], F(a["eps"]), a["pos"], a["axes"], a["axis"], a["table"], a["n"], a["rot"], a["il"],
           a["q_out"]]
    if write:
        return pq.lib().pqkv_qkv_norm_rope_write(
            a["q"], a["k"], a["v"], a["dt"], a["T"], a["hq"], a["hkv"], a["d"], a["qs"], a["ks"], a["vs"], *mid,
            a["slots"], a["cache"], a["scales"], a["oidx"], a["oval"], a["kv"], a["nb"], a["err"], None)
    return pq.lib().pqkv_qk_norm_rope(a["q"], a["k"], a["dt"], a["T"], a["hq"], a["hkv"], a["d"], a["qs"], a["ks"],
                                      *mid, a["k_out"], a["err"], None)


BAD_ROPE = [
    dict(dt=pq.FP8_E4M3), dict(T=-1), dict(hq=0), dict(d=96), dict(rot=60), dict(rot=72), dict(rot=-8), dict(il=2),
    dict(eps=float("nan")), dict(eps=-1.0), dict(axes=0), dict(axes=5), dict(n=0), dict(pos=None), dict(table=None),
    dict(table=A + 4), dict(qw=A + 8), dict(kw=A + 8), dict(axis=bytes([0, 1] * 16)), dict(q=None), dict(k=None),
    dict(q=A + 8), dict(qs=504), dict(qs=516), dict(ks=120), dict(q_out=None), dict(q_out=4 * A + 2), dict(err=None),
    dict(q_out=A + 64),             # into its own input, at another place
    dict(q_out=2 * A),              # over the keys
    dict(q_out=A, qs=1024),         # its own input, laid out otherwise
]


@pytest.mark.parametrize("bad", BAD_ROPE + [
    dict(hkv=-1), dict(k_out=None), dict(k_out=A), dict(k_out=4 * A), dict(hq=1 << 20, qs=1 << 26)], ids=str)
def test_norm_rope_refuses(bad):
    assert _rope(**bad) == pq.ERR_ARG


@pytest.mark.parametrize("bad", BAD_ROPE + [
    dict(hkv=0), dict(hkv=65536), dict(v=None), dict(vs=120), dict(slots=None), dict(cache=None), dict(cache=A + 8), dict(kv=9),
    dict(kv=pq.FP16), dict(nb=0), dict(nb=1 << 28), dict(kv=pq.FP8_E4M3, scales=None),
    dict(kv=pq.FP4_E2M1, oidx=None), dict(kv=pq.FP4_E2M1, oval=A + 2), dict(q_out=3 * A)], ids=str)
def test_norm_rope_write_refuses(bad):
    assert _rope(write=True, **bad) == pq.ERR_ARG


def test_no_tokens_is_no_work():
    nothing = dict(T=0, q=None, k=None, v=None, q_out=None, k_out=None, err=None, pos=None, table=None, slots=None,
                   cache=None)
    assert _rope(**nothing) == pq.OK
    assert _rope(write=True, **nothing) == pq.OK
    assert _rope(write=True, **dict(nothing, kv=9)) == pq.ERR_ARG


def _cross(**kw):
    a = dict(q=A, dt=pq.BF16, batch=2, most=4, hq=8, cu=A, cache=A, scales=A, oidx=A, oval=A, kv=pq.BF16, nb=16,
             hkv=2, d=64, tables=A, maxblk=4, lens=A, ranges=None, scale=0.1, out=A, err=A)
    a.update(kw)
    return pq.lib().pqkv_paged_cross_attention(
        a["q"], a["dt"], a["batch"], a["most"], a["hq"], a["cu"], a["cache"], a["scales"], a["oidx"], a["oval"],
        a["kv"], a["nb"], a["hkv"], a["d"], a["tables"], a["maxblk"], a["lens"], a["ranges"], F(a["scale"]), a["out"],
        a["err"], None)


@pytest.mark.parametrize("bad", [
    dict(dt=pq.FP16), dict(dt=pq.FP8_E4M3), dict(batch=-1), dict(most=0), dict(hq=0), dict(hq=7), dict(hq=6),
    dict(hkv=0), dict(d=96), dict(kv=7), dict(nb=0), dict(maxblk=0), dict(ranges=A + 4), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(q=None), dict(cu=None), dict(cache=None), dict(tables=None), dict(lens=None), dict(out=None), dict(err=None),
    dict(q=A + 2), dict(kv=pq.FP8_E4M3, scales=None), dict(kv=pq.FP4_E2M1, oval=None)], ids=str)
def test_cross_refuses(bad):
    assert _cross(**bad) == pq.ERR_ARG


def test_bindings_refuse_host_tensors():
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        pq.build_batch(i, i, i, i.view(2, 2), 4, i, i, i, i, i)
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pq.qk_norm_rope(x, x, None, None, x, x, i)
    c = pq.KVCache(pq.BF16, 1, 2, 64, torch.zeros(1, dtype=torch.uint8), None, None, None)
    with pytest.raises(ValueError):
        pq.qkv_norm_rope_write(x, x, x, None, None, x, i, c, i)
    with pytest.raises(ValueError):
        pq.paged_cross_attention(x, i, 1, c, i.view(2, 2), i, 1.0, x, i)


def test_binding_module_loads_and_refuses():
    """Its checks without a GPU: argument counts, types, tensors of the host (a device index of -1 matches none)."""
    m = pq._load_binding()
    x, i = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    for call, args in ((m.build_batch, (0, 0, i)), (m.build_batch, (0, 0) + (i,) * 10), (m.build_batch, (-1, 0) + (i,) * 10),
                       (m.qk_norm_rope, (0, 0, x, x, None, None, 1e-6, None, None, b"", False, x, x, i)),
                       (m.qk_norm_rope, (0, 0, 3, x, None, None, 1e-6, None, None, b"", False, x, x, i)),
                       (m.paged_cross_attention, ("a", 0) + (x,) * 17), (m.qkv_norm_rope_write, ())):
        with pytest.raises(ValueError):
            call(*args)


def test_plain_batch_agrees_with_the_host_slot_mapping():
    rng = np.random.default_rng(1)
    start, new = [0, 5, 16, 40], [3, 11, 0, 30]
    held = rng.permutation(100)[:40].reshape(4, 10)
    tables = np.where(np.arange(10)[None] < -(-np.array(start) // 16)[:, None], held, -1)
    need = sum(-(-(s + n) // 16) - -(-s // 16) for s, n in zip(start, new))
    ids = 100 + np.arange(need)
    t, slots, positions, cu, lens, err = ref.batch(start, new, ids, tables, 200, 50)
    assert err == 0 and list(cu) == [0, 3, 14, 14, 44] and list(lens) == [3, 16, 16, 70]
    np.testing.assert_array_equal(slots[:44], pq.build_slot_mapping(t.astype(np.int32), start, new))
    assert list(slots[44:]) == [-1] * 6 and list(positions[44:]) == [0] * 6


def test_plain_rotation_keeps_lengths_and_turns_by_differences():
    """Turning by p and then reading the inner product of two rows depends on the difference of their positions."""
    rng = np.random.default_rng(2)
    rot = 64
    angle = np.arange(50)[:, None] * 100.0 ** (-np.arange(rot // 2) / (rot // 2))
    table = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1)).float()
    x = torch.from_numpy(rng.standard_normal((1, 1, 64))).to(torch.bfloat16)
    y = torch.from_numpy(rng.standard_normal((1, 1, 64))).to(torch.bfloat16)
    for il in (False, True):
        at = lambda v, p: ref.norm_rope(v, None, 0, [p], b"", table, il)[0].ravel()  # noqa: E731
        np.testing.assert_allclose(at(x, 30) @ at(y, 11), at(x, 19) @ at(y, 0), rtol=1e-5, atol=1e-5)
        np.testing.assert_allclose(np.linalg.norm(at(x, 30)), np.linalg.norm(x.double().numpy()), rtol=1e-6)
    n, _ = ref.norm_rope(x, torch.ones(64), 0.0, None, b"", None, False)
    np.testing.assert_allclose((n ** 2).mean(), 1.0, rtol=1e-12)
