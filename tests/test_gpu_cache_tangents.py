"""Gradients that the cache's operators do not have are refused, not dropped."""
import pytest

from test_gpu_cache import DEV, gen, ints, msda, normal  # noqa: F401

torch = pytest.importorskip("torch")
import torch.autograd.forward_ad as fwAD  # noqa: E402

pytestmark = pytest.mark.gpu


def test_forward_mode(msda):  # noqa: F811
    g = gen(41)
    cache = msda.cache_create(4, 16, 2, 32)
    table, z = ints([0, 1]), ints(0)
    q, k, v = (normal(g, (1, 3, n, 32), torch.bfloat16) for n in (4, 2, 2))
    with fwAD.dual_level():
        dual = lambda x: fwAD.make_dual(x, torch.ones_like(x))           # noqa: E731
        for call in (lambda: msda.cache_attention(dual(q), cache, table, z), lambda: msda.cache_attention(q, cache, table, z, k, dual(v)),
                     lambda: msda.cache_attention(q, cache, table, z, dual(k), v), lambda: msda.cache_write(cache, dual(k), v, table, z),
                     lambda: msda.cache_write(cache, k, dual(v), table, z),
                     lambda: msda.cache_read(cache._replace(key=dual(cache.key)), table, z, 5),
                     lambda: msda.cache_attention(q, cache._replace(value=dual(cache.value)), table, z)):
            with pytest.raises(ValueError, match="no gradient"):
                call()
        msda.cache_write(cache, k, v, table, z)                          # no tangents: as ever
        out, _ = msda.cache_attention(q, cache, table, ints(3), k, v)
    assert out.isfinite().all()
