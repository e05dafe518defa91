"""Rows in which one key outweighs the others, over values of any size: what is added up stays within binary32."""
import pytest

import dense_reference as R
from test_gpu_cache import C, DEV, ints, msda  # noqa: F401
from test_gpu_cache_tail import tail

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("gap", [17.0, 25.0, 37.0])
@pytest.mark.parametrize("power", [-90, -60, 40, 70, 100])
@pytest.mark.parametrize("own", [0.0, 1.0])
@pytest.mark.parametrize("T", [1, 40])
def test_values_of_any_size(msda, T, own, power, gap, fmt, dtype):  # noqa: F811
    """The tail of 2599 keys lies up to 2^53 below one key, its values are 2^power, that key's 0 or the same; new tokens
    behind it."""
    B, S, M, N, D = 40, 2600, 8, 8, 32
    q, cache, table = tail(msda, fmt, dtype, B, T, S, M, N, D, gap, [100, 1500, S - 1])
    value = torch.full((B, S, N, D), 2.0 ** power, device=DEV)
    value[:, [100, 1500, S - 1]] *= own
    k, _ = msda.cache_read(cache, table, ints(*[S] * B), S, dtype=C.DT[dtype])
    msda.cache_write(cache, k, value.to(C.DT[dtype]), table, ints(*[0] * B))
    new = torch.zeros((B, T, N, D), device=DEV, dtype=C.DT[dtype])
    new_value = torch.full_like(new, 2.0 ** power)
    lengths = ints(*[S] * B)
    for args in ((), (new, new_value)):
        out, lse = msda.cache_attention(q, cache, table, lengths, *args, scale=1.0)
        for b in (0, B - 1):
            k, v = C.tokens(cache, table, b, S)
            ok = None
            if args:
                k, v = torch.cat((k, new[b].double())), torch.cat((v, new_value[b].double()))
                ok = torch.cat((torch.ones((T, S), dtype=torch.bool, device=DEV), torch.ones((T, T), dtype=torch.bool, device=DEV).tril()), 1)[None, None]
            want = R.attention(q[b:b + 1], k[None], (v * 2.0 ** -power)[None], None, ok, 1.0)
            value64, bound = want["out"]
            R.check(out[b:b + 1].double() * 2.0 ** -power, (value64, bound + 127 * 2.0 ** -33), "out")
            R.check(lse[b:b + 1], want["lse"], "lse")
