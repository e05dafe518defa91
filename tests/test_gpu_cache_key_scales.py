"""Keys whose scales lie far apart within a tile: a score is the product with what the cache stands for, whatever the
other keys of its tile are."""
import pytest

from test_gpu_cache import C, DEV, msda, normal, table_of, gen, ints  # noqa: F401
from test_gpu_cache_attention import compare, tree

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def keys(g, shape, dtype, far):
    """Three rows in ten (at random) have one channel of 2^far, which the queries do not have, and nothing else; the others are
    normal in channels 16 to 31."""
    B, S, N, D = shape
    k = torch.zeros(shape, device=DEV)
    k[..., 16:32] = torch.randn((B, S, N, 16), generator=g, device=DEV)
    big = torch.rand((B, S, N), generator=g, device=DEV) < 0.3
    k[big] = 0
    k[..., 3] = torch.where(big, 2.0 ** far, 0.0)
    return k.to(C.DT[dtype])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("far", [0, 7, 14, 20, 27, 40, 90])
def test_scales_within_a_tile(msda, far, T, fmt, dtype):  # noqa: F811
    B, S, M, N, D = 2, 700, 4, 2, 64
    g = gen(33)
    up = 1.0
    if dtype == "f16":                              # binary16 holds 2^27 apart only from 2^-12 to 2^15
        if far > 27:
            pytest.skip("beyond binary16")
        up = 2.0 ** (far // 2)
    cache = msda.cache_create(60, 32, N, D, C.FORMAT[fmt])
    table = table_of(g, B, 24, 60)
    k = (keys(g, (B, S, N, D), "f32", far) / up).to(C.DT[dtype])
    v = normal(g, (B, S, N, D), C.DT[dtype])
    msda.cache_write(cache, k, v, table, ints(0, 0))
    q = torch.zeros((B, T, M, D), device=DEV)
    q[..., 16:32] = torch.randn((B, T, M, 16), generator=g, device=DEV) * up
    q = q.to(C.DT[dtype])
    lengths = ints(S, 333)
    out, lse = compare(msda, q, cache, table, lengths)
    assert T == 1 or out.float().std(1).min() > 0
    key = (keys(g, (B, T, N, D), "f32", far) / up).to(C.DT[dtype])
    value = normal(g, (B, T, N, D), C.DT[dtype])
    compare(msda, q, cache, table, lengths, key, value)
    compare(msda, q, cache, table, lengths, key, value, mask=tree(g, B, T), counts=ints(T, max(1, T - 3)))
