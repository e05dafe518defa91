"""Gradients that the cache's operators do not have are refused, not dropped."""
import pytest

from test_gpu_cache import DEV, gen, ints, msda, normal  # noqa: F401

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def test_a_cache_that_requires_a_gradient(msda):  # noqa: F811
    g = gen(42)
    cache = msda.cache_create(4, 16, 2, 32)
    table, z = ints([0, 1]), ints(0)
    q, k, v = (normal(g, (1, 3, n, 32), torch.bfloat16) for n in (4, 2, 2))
    leaf = cache._replace(value=cache.value.clone().requires_grad_())
    for call in (lambda: msda.cache_write(leaf, k, v, table, z), lambda: msda.cache_read(leaf, table, z, 5),
                 lambda: msda.cache_attention(q, leaf, table, z)):
        with pytest.raises(ValueError, match="no gradient"):
            call()
        with torch.no_grad():
            call()
