"""The paged cache: rows written, quantised and read back, against the definition in 64 bits, bit for bit."""
import math

import pytest

torch = pytest.importorskip("torch")

import cache_reference as C  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def msda():
    import scale_deformable_attention_gb300 as m
    from scale_deformable_attention_gb300 import build

    build.build()
    m.device_errors()
    yield m
    assert m.device_errors() == 0


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def table_of(g, B, width, pages):
    return torch.randperm(pages, generator=g, device=DEV)[:B * width].view(B, width).int()


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def bits(x):
    return x.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[x.element_size()])


def filled(msda, g, pages, page, N, D, dtype, fmt):
    """A cache whose every byte is something."""
    cache = msda.cache_create(pages, page, N, D, C.FORMAT.get(fmt, C.DT[dtype]))
    for t in cache:
        if t is not None:
            b = bits(t)
            b.copy_(torch.randint(0, 120, b.shape, generator=g, device=DEV))
    return cache


FORMATS = ["same", "e4m3", "int8"]
SIZES = [
    # B, T, N, D, page, width
    (1, 1, 1, 16, 16, 1), (3, 5, 2, 48, 16, 3), (2, 33, 8, 64, 32, 4), (40, 1, 4, 128, 64, 2), (2, 200, 3, 80, 16, 20),
    (1, 1000, 1, 96, 256, 5), (5, 17, 5, 112, 1024, 1), (2, 4, 16, 32, 16, 2),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_write_and_read(msda, size, fmt, dtype):
    B, T, N, D, page, width = size
    g = gen(5)
    cache = filled(msda, g, B * width + 2, page, N, D, dtype, fmt)
    table = table_of(g, B, width, B * width + 2)
    room = width * page
    R_ = max(1, T * 2 // 3)
    key, value = normal(g, (B, T, N, D), C.DT[dtype]), normal(g, (B, T, N, D), C.DT[dtype]) * 30
    key[0, 0, 0] = 0
    for select in (False, True):
        before = [t.clone() if t is not None else None for t in cache]
        n = R_ if select else T
        sel = torch.rand((B, T), generator=g, device=DEV).argsort(1)[:, :n].int() if select else None
        counts = torch.randint(0, n + 1, (B,), generator=g, device=DEV).int()
        start = (torch.rand(B, generator=g, device=DEV) * (room - n + 1)).int()
        got = msda.cache_write(cache, key, value, table, start, counts=counts, select=sel)
        assert got is cache
        want = [t.clone() if t is not None else None for t in before]
        for b in range(B):
            at = torch.arange(int(counts[b]), device=DEV)
            src = at if sel is None else sel[b].long()[at]
            pos = at + int(start[b])
            block, place = table[b].long()[pos // page], pos % page
            for i, x in enumerate((key, value)):
                rows = x[b, src]
                if fmt == "same":
                    want[i][block, place] = rows
                else:
                    codes, byte = C.quantise(rows, C.FORMAT[fmt])
                    bits(want[i])[block, place] = bits(codes.to(torch.float32).to(C.FORMAT[fmt]))
                    want[2 + i][block, place] = byte.to(torch.uint8)
        for a, b in zip(cache, want):
            if a is not None:
                eq = bits(a) == bits(b)
                if a.dtype == torch.float8_e4m3fn:      # -0 and 0 are one value
                    eq |= (a.float() == 0) & (b.float() == 0)
                assert eq.all()
        # read back, in its own type and, quantised, in another
        for to in {dtype} | ({"f32", "bf16"} if fmt != "same" else set()):
            lengths = torch.randint(0, room + 1, (B,), generator=g, device=DEV).int()
            lengths[0] = room
            rows = room - 3 if room > 3 else room
            back = msda.cache_read(cache, table, lengths, rows, dtype=C.DT[to])
            for i, x in enumerate(back):
                assert x.shape == (B, rows, N, D) and x.dtype == C.DT[to]
                for b in range(B):
                    n = min(rows, int(lengths[b]))
                    assert torch.equal(x[b, :n], C.tokens(cache, table, b, n)[i].to(C.DT[to]))
                    assert not x[b, n:].any()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_rows_at_the_ends_of_the_range(msda, fmt):
    """Powers of two and their neighbours around the codes' largest value, subnormal and huge rows, infinities and NaN."""
    g = gen(6)
    most = C.MOST[C.FORMAT[fmt]]
    tops = [most * 2.0 ** e * f for e in (-120, -100, -60, -7, 0, 1, 60, 119) for f in (1.0, 1 + 2.0 ** -23, 1 - 2.0 ** -24, 0.5 + 2.0 ** -24)]
    tops = [t for t in tops if t < 3.4e38] + [3.4028234663852886e38, 1e-45, 1.17549435e-38, 2.0 ** -133]
    x = normal(g, (1, len(tops) + 4, 1, 32))
    x /= x.abs().amax(-1, keepdim=True)
    x[0, :len(tops), 0] *= torch.tensor(tops, dtype=torch.float64, device=DEV).float()[:, None]
    x[0, len(tops), 0, 3] = math.nan
    x[0, len(tops) + 1, 0, 31] = -math.inf
    x[0, len(tops) + 2] = 0
    x[0, len(tops) + 3] = torch.tensor([most, -most, most / 2, 0.5, 1.5, 2.5, -0.5, 3.5] * 4, device=DEV)
    cache = msda.cache_create(5, 16, 1, 32, C.FORMAT[fmt])
    table = ints([0, 1, 2, 3])
    n = x.shape[1]
    msda.cache_write(cache, x, -x, table, ints(7))
    codes, byte = C.quantise(x, C.FORMAT[fmt])
    k, v = msda.cache_read(cache, table, ints(7 + n), 7 + n, dtype=torch.float32)
    most = torch.finfo(torch.float32).max                     # a code that is rounded up past the range is read as its end
    want = C.stands_for(codes.float(), byte.to(torch.uint8)).clamp(-most, most).float()
    want[byte == 255] = math.nan
    assert torch.equal(torch.nan_to_num(k[:, 7:], nan=77.0), torch.nan_to_num(want, nan=77.0))
    assert torch.equal(torch.nan_to_num(v[:, 7:], nan=77.0), torch.nan_to_num(-want, nan=77.0))
    assert k[0, 7 + len(tops):9 + len(tops)].isnan().all()
    # half a step of the code at most
    fine = x[0].isfinite().all(-1, keepdim=True)
    off = (k[0, 7:].double() - x[0].double()).abs()
    scale = C.power(byte[0].int() - 127)[..., None]
    step = torch.maximum(x[0].double().abs() * 2.0 ** -4, 2.0 ** -10 * scale) if fmt == "e4m3" else scale / 2
    assert (off <= step)[fine.expand_as(off)].all()


def test_finite_rows_stay_finite(msda):
    x = torch.tensor([65504.0, -65504.0, 64512.0, 1.0] * 4, device=DEV, dtype=torch.float16).view(1, 1, 1, 16)
    for fmt in ("e4m3", "int8"):
        cache = msda.cache_create(1, 16, 1, 16, C.FORMAT[fmt])
        msda.cache_write(cache, x, -x, ints([0]), ints(0))
        for got, was in zip(msda.cache_read(cache, ints([0]), ints(1), 1, dtype=torch.float16), (x, -x)):
            assert got.isfinite().all() and (got.float() - was.float()).abs().max() <= 65504 * 2.0 ** -4


def test_places_that_do_not_exist(msda):
    """Pages, starts, lengths, counts and selections out of range: an error bit, nothing else touched."""
    g = gen(7)
    for fmt in FORMATS:
        cache = filled(msda, g, 6, 16, 2, 32, "bf16", fmt)
        key, value = normal(g, (3, 20, 2, 32), torch.bfloat16), normal(g, (3, 20, 2, 32), torch.bfloat16)
        table = torch.tensor([[0, -1], [1, 6], [2, 3]], dtype=torch.int32, device=DEV)
        before = [t.clone() if t is not None else None for t in cache]
        assert msda.device_errors() == 0
        msda.cache_write(cache, key, value, table, ints(0, 0, 20))       # a bad page each, and 12 rows behind the end
        assert msda.device_errors() == 8
        changed = (bits(cache.key) != bits(before[0])).any(-1).any(-1)
        assert changed[:2].all() and changed[3, 4:].all()
        changed[:2] = False
        changed[3, 4:] = False
        assert not changed.any()
        assert msda.device_errors() == 0
        sel = torch.zeros((3, 4), dtype=torch.int32, device=DEV)
        sel[0, 1], sel[2, 3] = 20, -1
        before = [t.clone() if t is not None else None for t in cache]
        ok = ints([4], [5], [0]).view(3, 1)
        msda.cache_write(cache, key, value, ok, ints(0, 0, -2), counts=ints(9, -1, 4), select=sel)
        assert msda.device_errors() == 8
        same = (bits(cache.key) == bits(before[0])).all(-1).all(-1)
        assert same[4].tolist() == [False, True, False, False] + [True] * 12 and same[5].all()  # a count of 9 is 4, of -1 none
        assert same[0].tolist() == [False] + [True] * 15                       # rows -2 and -1 are not, nor that of token -1
        k, _ = msda.cache_read(cache, table, ints(32, 40, -1), 32)
        assert msda.device_errors() == 8
        assert k[0, :16].any() and not k[0, 16:].any() and k[1, :16].any() and not k[1, 16:].any() and not k[2].any()


def test_far_pages(msda):
    """Offsets beyond 32 bits: pages behind 2^32 elements."""
    g = gen(8)
    pages, page, N, D = 135000, 256, 1, 128     # 4.4e9 elements of 8 bits
    cache = msda.cache_create(pages, page, N, D, torch.float8_e4m3fn)
    table = ints([pages - 1, 0], [pages - 2, pages // 2])
    key, value = normal(g, (2, 300, N, D), torch.bfloat16), normal(g, (2, 300, N, D), torch.bfloat16)
    msda.cache_write(cache, key, value, table, ints(0, 5))
    k, v = msda.cache_read(cache, table, ints(300, 305), 305)
    for b, first in ((0, 0), (1, 5)):
        for x, got in ((key, k), (value, v)):
            codes, byte = C.quantise(x[b], torch.float8_e4m3fn)
            assert torch.equal(got[b, first:first + 300], C.stands_for(codes.float(), byte.to(torch.uint8)).bfloat16())
    q = normal(g, (2, 1, 4, D), torch.bfloat16)
    want = C.attention(q, cache, table, ints(300, 305))
    out, lse = msda.cache_attention(q, cache, table, ints(300, 305))
    C.R.check(out, want["out"], "out")
    C.R.check(lse, want["lse"], "lse")


def test_any_layout(msda):
    """Token by token instead of head by head, pages of a larger pool, strided inputs: the same rows."""
    g = gen(9)
    B, T, N, D, page = 2, 40, 4, 64, 16
    big = torch.zeros((9, page, 2, N, 2 * D), device=DEV, dtype=torch.float16)
    cache = msda.PagedCache(big[:, :, 0, :, :D], big[:, :, 1, :, D:])
    plain = msda.cache_create(9, page, N, D, torch.float16)
    both = normal(g, (B, N, T, 2, D), torch.float16)
    key, value = both[:, :, :, 0].transpose(1, 2), both[:, :, :, 1].transpose(1, 2)
    odd = torch.zeros((B, T, N, D + 3), device=DEV, dtype=torch.float16)    # rows off 16 bytes are copied
    odd[..., 1:D + 1] = value
    table = table_of(g, B, 4, 9)
    wide = torch.full((B, 9), 99, device=DEV, dtype=torch.int32)
    wide[:, ::2][:, :4] = table
    start = ints(3, 0)
    msda.cache_write(cache, key, odd[..., 1:D + 1], wide[:, ::2][:, :4], start)
    msda.cache_write(plain, key.contiguous(), value.contiguous(), table, start)
    assert torch.equal(cache.key, plain.key) and torch.equal(cache.value, plain.value)
    q = normal(g, (B, 3, 8, D), torch.float16)
    lengths = ints(43, 40)
    assert all(torch.equal(a, b) for a, b in zip(msda.cache_attention(q, cache, table, lengths),
                                                 msda.cache_attention(q, plain, table, lengths)))


def test_nothing_to_do(msda):
    cache = msda.cache_create(0, 16, 2, 32)
    z = torch.zeros((2, 0, 2, 32), device=DEV, dtype=torch.bfloat16)
    table = torch.zeros((2, 0), device=DEV, dtype=torch.int32)
    msda.cache_write(cache, z, z, table, ints(0, 0))
    k, v = msda.cache_read(cache, table, ints(0, 0), 5)
    assert not k.any() and not v.any() and k.shape == (2, 5, 2, 32)
    k, _ = msda.cache_read(cache, table[:0], ints(), 5)
    assert k.shape == (0, 5, 2, 32)
    out, lse = msda.cache_attention(z, cache, table, ints(0, 0))
    assert out.shape == (2, 0, 64) and lse.shape == (2, 2, 0)
    q = torch.ones((2, 3, 4, 32), device=DEV, dtype=torch.bfloat16)
    out, lse = msda.cache_attention(q, cache, table, ints(0, 0))
    assert not out.any() and (lse == -math.inf).all()
    out, lse = msda.cache_attention(q, cache, table, ints(0, 0), q[:, :, :2], q[:, :, :2])
    assert (out == 1).all()
