"""A cache of no pages under a table of some width: nothing is written, read or seen, and the error bit tells of lengths above 0."""
import ctypes
import math

import pytest

from test_gpu_cache import C, DEV, FORMATS, gen, ints, msda, normal  # noqa: F401
from test_gpu_cache_attention import compare

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 17, 40, 300])
def test_attention(msda, T, fmt, dtype):  # noqa: F811
    g = gen(30)
    N, D = 2, 64
    cache = msda.cache_create(0, 16, N, D, C.FORMAT.get(fmt, C.DT[dtype]))
    table = torch.randint(-3, 9, (2, 40), generator=g, device=DEV).int()
    q, key, value = (normal(g, (2, T, n, D), C.DT[dtype]) for n in (4, 2, 2))
    assert msda.device_errors() == 0
    for lengths in (ints(0, 0), ints(640, 3)):
        out, lse = msda.cache_attention(q, cache, table, lengths)
        assert not out.any() and (lse == -math.inf).all()
        assert msda.device_errors() == (8 if lengths.any() else 0)
        got = msda.cache_attention(q, cache, table, lengths, key, value)
        assert msda.device_errors() == (8 if lengths.any() else 0)
        want = compare(msda, q, cache, table, ints(0, 0), key, value)       # the new tokens alone
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("fmt", FORMATS)
def test_write_and_read(msda, fmt):  # noqa: F811
    g = gen(30)
    cache = msda.cache_create(0, 16, 2, 32, C.FORMAT.get(fmt, torch.bfloat16))
    table = torch.randint(-3, 9, (2, 40), generator=g, device=DEV).int()
    x = normal(g, (2, 20, 2, 32), torch.bfloat16)
    assert msda.device_errors() == 0
    msda.cache_write(cache, x, x, table, ints(0, 7))
    assert msda.device_errors() == 8
    msda.cache_write(cache, x, x, table, ints(0, 7), counts=ints(0, 0))
    assert msda.device_errors() == 0
    for lengths in (ints(0, 0), ints(640, 3)):
        k, v = msda.cache_read(cache, table, lengths, 50)
        assert not k.any() and not v.any()
        assert msda.device_errors() == (8 if lengths.any() else 0)


@pytest.mark.parametrize("T", [3, 40])
def test_null_pointers(msda, T):  # noqa: F811
    """The C calls with no cache and no table at all."""
    from scale_deformable_attention_gb300 import _lib

    B, M, N, D, width = 2, 4, 2, 32, 4
    rows = lambda n: (T * n * D, n * D, D)                           # noqa: E731
    p = _lib.cache_problem(B, T, M, N, D, T, 0, 16, width, width * 16, *(0,) * 12, width, *rows(M), *rows(N), *rows(N), 0, 0, 0)
    q, k, v = (normal(gen(30), (B, T, n, D), torch.bfloat16) for n in (M, N, N))
    lengths = ints(64, 5)
    out, lse = torch.empty_like(q), torch.empty((B, M, T), device=DEV)
    at = lambda t: ctypes.c_void_p(t.data_ptr())                     # noqa: E731
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    lib = _lib.lib()
    none = (None,) * 5
    assert lib.msda_cache_attention_workspace_size(2, 0, p) == 0
    assert lib.msda_cache_attention(2, 0, p, D ** -0.5, at(q), *none, at(lengths), at(k), at(v), None, None, at(out), at(lse), None, 0, st) == 0
    want = msda.cache_attention(q, msda.cache_create(0, 16, N, D), torch.zeros((B, width), device=DEV, dtype=torch.int32), ints(0, 0), k, v)
    assert torch.equal(out.view(B, T, M * D), want[0]) and torch.equal(lse, want[1])
    assert lib.msda_cache_write(2, 0, p, at(k), at(v), None, at(lengths), None, None, None, None, None, None, st) == 0
    assert lib.msda_cache_read(2, 0, p, *none, at(lengths), at(k), at(v), st) == 0
    assert not k.any() and not v.any() and msda.device_errors() == 8
