"""The Python module of the serving-step calls is used, and kept by a build, only
with the Python and torch that it was compiled for."""
import pytest

pq = pytest.importorskip("paged_quantized_kv_cache_b200")

from paged_quantized_kv_cache_b200 import build  # noqa: E402


def test_the_built_module_is_for_this_python_and_torch():
    assert pq._load_binding().BUILT_FOR == build.binding_target()
    assert build._binding_fits()


@pytest.mark.parametrize("other", ["for python 3.12, torch 2.11.0", "for python 3.9, torch 2.11.0+cu128"])
def test_a_module_for_another_one_is_refused_and_built_anew(monkeypatch, other):
    monkeypatch.setattr(build, "binding_target", lambda: other)
    assert build._binding_stale()
    with pytest.raises(ImportError, match="another torch|built for"):
        pq._load_binding()
