"""The rotary calls refuse an output that shares memory with anything but its own
input: on the host, before a launch."""
import pytest
import torch

from tests.test_step_refusals import A, _rope

pq = pytest.importorskip("paged_quantized_kv_cache_b200")

# everything apart, by A each; q_out of 4 tokens, 8 heads of 64: 4096 bytes
APART = dict(q=A, k=2 * A, v=3 * A, q_out=4 * A, k_out=5 * A, cache=6 * A, pos=7 * A, table=8 * A, qw=9 * A, kw=10 * A,
             slots=11 * A, scales=12 * A, oidx=13 * A, oval=14 * A, err=15 * A, axes=3)
BOTH = [("pos", -32), ("pos", 4092), ("table", -16 * 64 * 4 + 16), ("table", 4080), ("qw", -240), ("qw", 4080), ("kw", 16),
        ("err", 4092)]


@pytest.mark.parametrize("array,at", BOTH, ids=str)
def test_queries_over_another_array(array, at):
    bad = dict(APART, **{array: 4 * A + at})
    assert _rope(**bad) == pq.ERR_ARG
    assert _rope(write=True, **bad) == pq.ERR_ARG


@pytest.mark.parametrize("array,at", [("pos", 1020), ("table", 16), ("qw", 1008), ("kw", -240), ("err", 0)], ids=str)
def test_keys_over_another_array(array, at):
    assert _rope(**dict(APART, **{array: 5 * A + at})) == pq.ERR_ARG


@pytest.mark.parametrize("kv,array,at", [
    (pq.BF16, "slots", 4092), (pq.BF16, "cache", -64 * 2 * 2 * 16 * 128 + 16), (pq.FP8_E4M3, "cache", 4080),
    (pq.FP8_E4M3, "scales", -64 * 2 * 16 + 16), (pq.FP4_E2M1, "scales", 0), (pq.FP4_E2M1, "oidx", -64 * 2 * 16 + 16),
    (pq.FP4_E2M1, "oval", 4080)], ids=str)
def test_queries_over_the_cache(kv, array, at):
    assert _rope(write=True, **dict(APART, kv=kv, **{array: 4 * A + at})) == pq.ERR_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="the arguments are addresses that no kernel may see")
@pytest.mark.parametrize("good", [
    dict(), dict(pos=4 * A - 48), dict(pos=4 * A + 4096), dict(table=4 * A - 16 * 64 * 4), dict(qw=4 * A - 256), dict(qw=4 * A + 4096),
    dict(q_out=A), dict(rot=0, pos=4 * A, table=4 * A), dict(kv=pq.BF16, scales=4 * A)], ids=str)
def test_arrays_side_by_side_and_in_place(good):
    a = dict(APART, **good)
    assert _rope(**a) == pq.ERR_CUDA  # past the checks: there is no device
    assert _rope(write=True, **a) == pq.ERR_CUDA
