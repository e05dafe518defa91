"""Caches that another program filled: scale bytes of 255 over codes that are not 0, e4m3 codes that are NaN."""
import pytest

from test_gpu_cache import C, DEV, msda, normal, table_of, gen, ints  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def pool(msda, g, fmt, B, S, N, D):  # noqa: F811
    cache = msda.cache_create(40, 16, N, D, C.FORMAT[fmt])
    table = table_of(g, B, 16, 40)
    k, v = (normal(g, (B, S, N, D), torch.bfloat16) for _ in range(2))
    msda.cache_write(cache, k, v, table, ints(*[0] * B))
    return cache, table


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("T", [1, 40])
def test_byte_255_is_a_row_of_nan(msda, T, fmt, dtype):  # noqa: F811
    B, S, M, N, D = 2, 200, 4, 2, 32
    g = gen(34)
    cache, table = pool(msda, g, fmt, B, S, N, D)
    lengths = ints(S, S)
    cache.key_scale[table[0, 3].long(), 5, 0] = 255            # sequence 0, token 53, head 0
    cache.value_scale[table[1, 7].long(), 2, 1] = 255          # sequence 1, token 114, head 1
    back = msda.cache_read(cache, table, lengths, S, dtype=C.DT[dtype])
    for x, at in zip(back, ((0, 53, 0), (1, 114, 1))):
        nan = torch.zeros_like(x, dtype=torch.bool)
        nan[at] = True
        assert torch.equal(x.isnan(), nan)
    q = normal(g, (B, T, M, D), C.DT[dtype])
    out, lse = msda.cache_attention(q, cache, table, lengths)
    out = out.view(B, T, M, D)
    assert lse[0, :2].isnan().all() and lse[0, 2:].isfinite().all() and lse[1].isfinite().all()
    assert out[0, :, :2].isnan().all() and out[0, :, 2:].isfinite().all()
    assert out[1, :, 2:].isnan().all() and out[1, :, :2].isfinite().all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("byte", [27, 127, 134, 140, 246])
def test_codes_of_nan_are_read_as_nan(msda, byte, dtype):  # noqa: F811
    """Under any scale; what else the row has is code * scale, at most the type's largest value."""
    g = gen(35)
    cache, table = pool(msda, g, "e4m3", 1, 50, 1, 16)
    for codes, scale in ((cache.key, cache.key_scale), (cache.value, cache.value_scale)):
        codes.view(torch.uint8)[table[0, 1].long(), 4, 0, 7] = 0x7f
        codes.view(torch.uint8)[table[0, 1].long(), 4, 0, 8] = 0xff
        scale[table[0, 1].long(), 4, 0] = byte
    most = torch.finfo(C.DT[dtype]).max
    want = C.tokens(cache, table, 0, 50)
    for x, y in zip(msda.cache_read(cache, table, ints(50), 50, dtype=C.DT[dtype]), want):
        y = y.clamp(-most, most).to(C.DT[dtype])               # clamp keeps NaN
        assert int(x.isnan().sum()) == 2 and x[0, 20, 0, 7].isnan() and x[0, 20, 0, 8].isnan()
        assert torch.equal(x[0].nan_to_num(nan=7.0), y.nan_to_num(nan=7.0))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T", [1, 40])
def test_codes_of_nan_are_attended_to_as_nan(msda, T, dtype):  # noqa: F811
    g = gen(36)
    cache, table = pool(msda, g, "e4m3", 1, 50, 2, 16)
    cache.value.view(torch.uint8)[table[0, 1].long(), 4, 0, 7] = 0x7f
    cache.key.view(torch.uint8)[table[0, 1].long(), 9, 1, 3] = 0xff
    q = normal(g, (1, T, 4, 16), C.DT[dtype])
    out, lse = msda.cache_attention(q, cache, table, ints(50))
    out = out.view(1, T, 4, 16)
    assert out[0, :, :2, 7].isnan().all() and int(out[0, :, :2].isnan().sum()) == 2 * T and lse[0, :2].isfinite().all()
    assert out[0, :, 2:].isnan().all() and lse[0, 2:].isnan().all()
