"""Values whose scales lie far apart within a tile: what a row attends to counts, whatever the tile's others are."""
import pytest

import dense_reference as R
from test_gpu_cache import C, DEV, gen, ints, msda, normal, table_of  # noqa: F401
from test_gpu_cache_attention import compare

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("T", [1, 40, 150])
@pytest.mark.parametrize("far", [12, 18, 22, 23, 24, 25, 26, 27, 28, 36])
def test_a_small_value_next_to_large_ones(msda, far, T, fmt, dtype):  # noqa: F811
    """Query t looks at one token, whose value is 2^far below the others', which have 60 exp(-32) = 2^-40 of the row together.

    A code is rounded to half of binary16's smallest step, 2^-25, in units of the tile's largest scale over 2^7 (e4m3) or 2^5
    (int8), and that scale is at most 2 / 448 or 2 / 127 of the largest value: 2^-36 of it and less.  With the others' share
    2^-35 holds both, as far as a scale down to 2^-24 of that unit holds rows, 2^28 below the largest (e4m3) and 2^26 (int8);
    beyond, rows count as 0, 2^-29 of the largest.
    """
    B, S, M, N, D = 2, 60, 4, 2, 64
    if dtype == "f16" and far > 26:
        pytest.skip("beyond binary16")
    g = gen(44)
    cache = msda.cache_create(20, 16, N, D, C.FORMAT[fmt])
    table = table_of(g, B, 4, 20)
    k = torch.zeros((B, S, N, D), device=DEV)
    k[:, torch.arange(S), :, torch.arange(S)] = 16.0               # each token a channel of its own
    v = normal(g, (B, S, N, D)) * (2.0 ** 13 if dtype == "f16" else 2.0 ** 20)
    small = torch.arange(3, S, 7, device=DEV)
    v[:, small] *= 2.0 ** -far
    msda.cache_write(cache, k.to(C.DT[dtype]), v.to(C.DT[dtype]), table, ints(0, 0))
    q = torch.zeros((B, T, M, D), device=DEV)
    at = small[torch.arange(T, device=DEV) % len(small)]
    q[:, torch.arange(T), :, at] = 2.0
    q = q.to(C.DT[dtype])
    out, lse = msda.cache_attention(q, cache, table, ints(S, S), scale=1.0)
    part = 2.0 ** -35 if far <= (28 if fmt == "e4m3" else 26) else 2.0 ** -29
    for b in range(B):
        k, v = C.tokens(cache, table, b, S)
        want = R.attention(q[b:b + 1], k[None], v[None], scale=1.0)
        value, bound = want["out"]
        R.check(out[b:b + 1], (value, bound + part * float(v.abs().max())), "out")
        R.check(lse[b:b + 1], want["lse"], "lse")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("top", [65504.0, 65280.0, 32768.0, 1.0])
def test_largest_new_values(msda, top, fmt, dtype):  # noqa: F811
    """New tokens at the end of binary16's range (and of a power of two) over codes."""
    B, T, M, N, D = 2, 40, 4, 2, 32
    g = gen(45)
    cache = msda.cache_create(20, 16, N, D, C.FORMAT[fmt])
    table = table_of(g, B, 4, 20)
    x = normal(g, (B, 50, N, D), C.DT[dtype])
    msda.cache_write(cache, x, x, table, ints(0, 0))
    q = normal(g, (B, T, M, D), C.DT[dtype])
    key = normal(g, (B, T, N, D))
    key[:, ::3, :, 2] = top
    value = torch.rand((B, T, N, D), generator=g, device=DEV) * top
    value[:, ::2, :, 5] = top
    value[:, 1::2, :, 9] = -top
    compare(msda, q, cache, table, ints(50, 0), key.to(C.DT[dtype]), value.to(C.DT[dtype]), scale=1.0 / top)
