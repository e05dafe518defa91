"""Queries at the end of a type's range over a quantised cache."""
import pytest

from test_gpu_cache import C, gen, ints, msda, normal, table_of  # noqa: F401
from test_gpu_cache_attention import compare

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("power", [100, 115, 117, 125])
def test_large_queries_over_codes(msda, power, T, fmt, dtype):  # noqa: F811
    """Queries near the end of the range over keys near its other end."""
    B, S, M, N, D = 2, 300, 4, 2, 32
    g = gen(40)
    cache = msda.cache_create(50, 16, N, D, C.FORMAT[fmt])
    table = table_of(g, B, 20, 50)
    k = normal(g, (B, S, N, D)) * 2.0 ** -90
    msda.cache_write(cache, k.to(C.DT[dtype]), normal(g, (B, S, N, D), C.DT[dtype]), table, ints(0, 0))
    q = (normal(g, (B, T, M, D)) * 2.0 ** power).to(C.DT[dtype])
    compare(msda, q, cache, table, ints(S, 77), scale=2.0 ** (88 - power))
