"""The paged cache's C ABI and binding on the host, without a GPU: refusals and
sizes of workspaces.  No call here reaches a launch: each fails validation first."""
import pytest

torch = pytest.importorskip("torch")
FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    from scale_deformable_attention_gb300 import _lib, build

    build.build()
    return _lib.lib()


def problem(B=2, T=3, M=4, N=2, D=32, source=3, pages=9, page=16, width=4, longest=64, ck=None, cv=None, ks=None, vs=None,
            ts=None, q=None, k=None, v=None, ms=(0, 0), ss=0):
    from scale_deformable_attention_gb300._lib import cache_problem

    pool = (N * page * D, D, page * D)
    scales = (N * page, 1, page)
    rows = lambda heads: (T * heads * D, heads * D, D)              # noqa: E731
    return cache_problem(B, T, M, N, D, source, pages, page, width, longest, *(ck or pool), *(cv or pool), *(ks or scales),
                        *(vs or scales), width if ts is None else ts, *(q or rows(M)), *(k or rows(N)), *(v or rows(N)), *ms, ss)


def write(lib, p, dt=2, fmt=1, **ptrs):
    a = dict.fromkeys(("key", "value", "table", "start"), FAKE) | {"counts": None, "select": None}
    a |= dict.fromkeys(("cache_key", "cache_value", "key_scale", "value_scale"), FAKE) | ptrs
    return lib.msda_cache_write(dt, fmt, p, *a.values(), None)


def read(lib, p, dt=2, fmt=1, **ptrs):
    a = dict.fromkeys(("cache_key", "cache_value", "key_scale", "value_scale", "table", "lengths", "key", "value"), FAKE) | ptrs
    return lib.msda_cache_read(dt, fmt, p, *a.values(), None)


def attend(lib, p, dt=2, fmt=1, scale=1.0, ws=None, n=0, **ptrs):
    a = dict.fromkeys(("query", "cache_key", "cache_value", "key_scale", "value_scale", "table", "lengths", "key", "value"), FAKE)
    a |= {"mask": None, "counts": None, "out": FAKE, "lse": FAKE} | ptrs
    return lib.msda_cache_attention(dt, fmt, p, scale, *a.values(), ws, n, None)


def msg(lib):
    return lib.msda_last_error().decode()


@pytest.mark.parametrize("call", [write, read, attend])
@pytest.mark.parametrize("kw,status,text", [
    (dict(B=-1), 1, "negative"), (dict(T=-1), 1, "negative"), (dict(source=-1), 1, "negative"), (dict(pages=-1), 1, "negative"),
    (dict(width=-1), 1, "negative"), (dict(longest=-1), 1, "negative"), (dict(N=0), 1, "at least 1"), (dict(D=0), 1, "at least 1"),
    (dict(D=40), 2, "channels"), (dict(D=144), 2, "channels"), (dict(page=8), 2, "power of two"), (dict(page=48), 2, "power of two"),
    (dict(page=0), 2, "power of two"), (dict(longest=65), 1, "longest=65"), (dict(width=1 << 27), 2, "too large"),
    (dict(B=1 << 31), 2, "too large"), (dict(pages=1 << 31), 2, "too large"), (dict(N=70000, M=70000), 2, "too large"),
    (dict(ck=(-1, 1, 1)), 1, "negative stride"), (dict(vs=(1, -1, 1)), 1, "negative stride"), (dict(ts=-4), 1, "negative stride"),
    (dict(q=(1, 1, -1)), 1, "negative stride"), (dict(ms=(0, -1)), 1, "negative stride"), (dict(ss=-1), 1, "negative stride"),
])
def test_sizes_are_checked(lib, call, kw, status, text):
    assert call(lib, problem(**kw)) == status
    assert text in msg(lib)


@pytest.mark.parametrize("call", [write, read, attend])
def test_arguments_are_checked(lib, call):
    p = problem()
    assert call(lib, p, dt=5) == 1 and "dtype" in msg(lib)
    assert call(lib, p, fmt=3) == 1 and "format" in msg(lib)
    assert call(lib, None) == 1 and "problem" in msg(lib)
    for name in ("cache_key", "cache_value", "key", "value"):
        assert call(lib, p, **{name: None}) == 1 and "NULL" in msg(lib)
        assert call(lib, p, **{name: FAKE + 8}) == 3
    for name in ("key_scale", "value_scale", "table"):
        assert call(lib, p, **{name: None}) == 1 and "NULL" in msg(lib)
    assert call(lib, p, table=FAKE + 2) == 3
    assert call(lib, problem(ck=(1024, 24, 512))) == 3 and "cache key" in msg(lib)      # 24 codes are no whole vectors
    assert call(lib, problem(cv=(1000, 32, 512))) == 3 and "cache value" in msg(lib)
    name = "start" if call is write else "lengths"
    assert call(lib, p, **{name: None}) == 1 and name in msg(lib)
    assert call(lib, p, **{name: FAKE + 1}) == 3


def test_write_refuses(lib):
    assert write(lib, problem(source=2)) == 1 and "without select" in msg(lib)
    assert write(lib, problem(), select=FAKE + 2) == 3
    assert write(lib, problem(), counts=FAKE + 2) == 3
    assert write(lib, problem(k=(100, 32, 32))) == 3 and "key" in msg(lib)
    assert write(lib, problem(T=1 << 29, source=1 << 29, N=8, M=8, B=0)) == 2 and "too many" in msg(lib)


def test_attention_refuses(lib):
    assert attend(lib, problem(M=3)) == 1 and "divide" in msg(lib)
    assert attend(lib, problem(source=2)) == 1 and "source" in msg(lib)
    assert attend(lib, problem(source=0), mask=FAKE) == 1 and "mask" in msg(lib)
    assert attend(lib, problem(B=1 << 20, T=1 << 20, source=1 << 20)) == 2 and "too many" in msg(lib)
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert attend(lib, problem(), scale=scale) == 1 and "scale" in msg(lib)
    for name in ("query", "out", "lse"):
        assert attend(lib, problem(), **{name: None}) == 1 and name in msg(lib)
        assert attend(lib, problem(), **{name: FAKE + 2}) == 3
    long = problem(width=4000, longest=64000)
    need = lib.msda_cache_attention_workspace_size(2, 1, long)
    assert need > 0
    for ws, n in ((None, 0), (FAKE, need - 1), (FAKE + 16, need)):
        assert attend(lib, long, ws=ws, n=n) == 4 and "workspace" in msg(lib)


def test_workspaces(lib):
    size = lib.msda_cache_attention_workspace_size
    assert size(2, 1, problem(D=33)) == 0 and size(2, 1, problem(B=0, width=4000, longest=64000)) == 0
    assert size(2, 1, problem()) == 0                                       # 64 tokens: nothing to join
    a = size(2, 1, problem(width=4000, longest=64000))
    assert a % 4 == 0 and a <= 304 * 3 * 32 * 33 * 4 and size(2, 1, problem(width=4000, longest=400)) <= a


def test_nothing_to_do(lib):
    none = dict.fromkeys(("key", "value", "cache_key", "cache_value", "key_scale", "value_scale", "table"))
    for kw in (dict(B=0), dict(T=0, source=0)):
        assert write(lib, problem(**kw), start=None, **none) == 0
        assert read(lib, problem(**kw), lengths=None, **none) == 0
        assert attend(lib, problem(**kw), lengths=None, query=None, out=None, lse=None, **none) == 0


def test_binding_refuses_on_the_host():
    import scale_deformable_attention_gb300 as msda

    for kw in (dict(page=24), dict(page=8), dict(channels=40), dict(channels=144), dict(heads=0), dict(pages=-1)):
        with pytest.raises(ValueError):
            msda.cache_create(**({"pages": 2, "page": 16, "heads": 1, "channels": 32, "device": "cpu"} | kw))
    with pytest.raises(TypeError, match="cache dtype"):
        msda.cache_create(2, 16, 1, 32, torch.float64, "cpu")
    cache = msda.cache_create(2, 16, 1, 32, torch.int8, "cpu")
    assert cache.key.shape == (2, 16, 1, 32) and cache.key_scale.shape == (2, 16, 1) and cache.key_scale.dtype == torch.uint8
    x, i = torch.zeros(1, 1, 1, 32), torch.zeros(1, dtype=torch.int32)
    for call in (lambda: msda.cache_write(cache, x, x, i[None], i), lambda: msda.cache_read(cache, i[None], i, 3),
                 lambda: msda.cache_attention(x, cache, i[None], i)):
        with pytest.raises(ValueError, match="CUDA tensors only"):
            call()
