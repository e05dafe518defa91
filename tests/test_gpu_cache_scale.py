"""The smallest scales that a call over the paged cache may give."""
import pytest

from test_gpu_cache import C, FORMATS, msda, normal  # noqa: F401
from test_gpu_cache_attention import compare, made, tree

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("scale", [1e-300, 1e-46, 1e-44, 1e-20])
def test_scales_that_binary32_hardly_holds(msda, scale, T, fmt, dtype):  # noqa: F811
    """Scores are 0 to binary32: what a query sees weighs the same, the rest nothing."""
    g, cache, table, lengths = made(msda, 31, dtype, fmt, 3, 700, 2, 64, 32, [700, 0, 333])
    q, key, value = (normal(g, (3, T, n, 64), C.DT[dtype]) for n in (4, 2, 2))
    compare(msda, q, cache, table, lengths, scale=scale)
    compare(msda, q, cache, table, lengths, key, value, scale=scale)
    compare(msda, q, cache, table, lengths, key, value, mask=tree(g, 3, T), scale=scale)
