"""The serving-step calls refuse cache arrays that are smaller than the cache's
numbers make them, before anything is launched: without a GPU, on tensors that
have a device, a type and a shape but no memory."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

pq = pytest.importorskip("paged_quantized_kv_cache_b200")

NB, HKV, D, T = 6, 2, 64, 4
FORMATS = {pq.BF16: 1, pq.FP8_E4M3: 2, pq.FP8_E5M2: 2, pq.FP4_E2M1: 4}  # arrays that each has
NAMES = ("cache", "scales", "outliers_idx", "outliers_val")


def _calls(sizes, kv_dtype, nb=NB):
    """What the two calls that take a cache answer: the library's status (it refuses null pointers) or an error."""
    m = pq._binding_module or pq._load_binding()
    with FakeTensorMode():
        new = lambda *n, dtype=torch.int32: torch.empty(*n, dtype=dtype, device="cuda:0")  # noqa: E731
        cache = [new(n, dtype=torch.uint8) if n else None for n in sizes] + [kv_dtype, nb, HKV, D]
        q, kv = new(T, 8, D, dtype=torch.bfloat16), new(T, HKV, D, dtype=torch.bfloat16)
        yield lambda: m.paged_cross_attention(0, 0, q, new(3), 4, *cache, new(2, 3), new(2), None, 1.0, q, new(1))
        yield lambda: m.qkv_norm_rope_write(0, 0, q, kv, kv, None, None, 1e-6, None, None, b"", False, q, new(T), *cache,
                                            new(1))


@pytest.mark.filterwarnings("ignore")
@pytest.mark.parametrize("kv_dtype,array", [(f, i) for f, n in FORMATS.items() for i in range(n)])
def test_a_short_array_is_refused(kv_dtype, array):
    sizes = list(pq.cache_layout(kv_dtype, NB, HKV, D))
    for call in _calls(sizes, kv_dtype):
        assert call() == pq.ERR_ARG
    sizes[array] -= 1
    for call in _calls(sizes, kv_dtype):
        with pytest.raises(ValueError, match=NAMES[array]):
            call()


@pytest.mark.filterwarnings("ignore")
@pytest.mark.parametrize("kv_dtype", FORMATS)
def test_a_count_of_blocks_that_the_arrays_do_not_hold_is_refused(kv_dtype):
    sizes = pq.cache_layout(kv_dtype, NB, HKV, D)
    for nb in (NB + 1, 2 ** 26):
        for call in _calls(sizes, kv_dtype, nb):
            with pytest.raises(ValueError, match="cache"):
                call()
    for nb in (NB - 1, 1, 0):  # fewer blocks than there are, and a count that the library refuses
        for call in _calls(sizes, kv_dtype, nb):
            assert call() == pq.ERR_ARG
