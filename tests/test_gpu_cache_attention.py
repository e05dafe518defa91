"""Attention of new tokens over the paged cache against the dense definition in 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")

import cache_reference as C  # noqa: E402
from test_gpu_cache import DEV, FORMATS, gen, ints, msda, normal, table_of  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def made(msda, seed, dtype, fmt, B, S, N, D, page, lengths=None):  # noqa: F811
    """A cache that holds `lengths` (S: all) tokens of each sequence, what lies behind being NaN; scales differ by row."""
    g = gen(seed)
    width = max(1, -(-S // page))
    pages = B * width + 2
    cache = msda.cache_create(pages, page, N, D, C.FORMAT.get(fmt, C.DT[dtype]))
    table = table_of(g, B, width, pages)
    lengths = ints(*([S] * B if lengths is None else lengths))
    x = [normal(g, (B, S, N, D), C.DT[dtype]) for _ in range(2)]
    x[1] *= torch.exp2(torch.randint(-3, 4, (B, S, N, 1), generator=g, device=DEV).float()).to(x[1].dtype)
    poison(cache)
    msda.cache_write(cache, x[0], x[1], table, torch.zeros_like(lengths), counts=lengths)
    unused = torch.arange(width, device=DEV)[None] * page >= lengths[:, None]
    table[unused] = -7
    return g, cache, table, lengths


def poison(cache):
    for t in cache:
        if t is None:
            continue
        if t.element_size() == 1:
            t.view(torch.uint8).fill_(0x7f if t.dtype == torch.float8_e4m3fn else 255)
        else:
            t.fill_(math.nan)


def tree(g, B, T):
    sees = torch.eye(T, dtype=torch.bool, device=DEV).repeat(B, 1, 1)
    for b in range(B):
        up = torch.randint(0, 4, (T,), generator=g, device=DEV).tolist()
        for t in range(1, T):
            if t - 1 - up[t] >= 0:
                sees[b, t] |= sees[b, t - 1 - up[t]]
    return sees


def compare(msda, q, cache, table, lengths, key=None, value=None, **kw):  # noqa: F811
    want = C.attention(q, cache, table, lengths, key, value, kw.get("mask"), kw.get("counts"), kw.get("scale"))
    out, lse = msda.cache_attention(q, cache, table, lengths, key, value, **kw)
    C.R.check(out, want["out"], "out")
    C.R.check(lse, want["lse"], "lse")
    return out, lse


SIZES = [
    # B, T, S, M, N, D, page
    (1, 1, 1, 1, 1, 16, 16), (2, 1, 300, 8, 8, 32, 16), (3, 1, 2047, 8, 2, 64, 64), (1, 1, 20011, 16, 4, 128, 256),
    (40, 1, 130, 4, 2, 48, 16), (2, 5, 777, 6, 2, 80, 32), (2, 16, 1500, 4, 4, 128, 128), (2, 17, 515, 8, 8, 64, 32),
    (1, 31, 900, 8, 4, 96, 64), (2, 64, 1111, 8, 2, 128, 64), (1, 130, 257, 4, 2, 64, 16), (2, 3, 0, 4, 2, 112, 16),
    (1, 2, 4100, 32, 1, 64, 1024), (1, 300, 1000, 4, 4, 32, 256), (5, 8, 40, 2, 1, 16, 32),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("new", ["none", "chain", "tree", "ragged"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_sizes(msda, size, new, fmt, dtype):  # noqa: F811
    B, T, S, M, N, D, page = size
    lengths = [S if b == 0 else (S * ((b * 5 + 3) % 8)) // 7 for b in range(B)]
    g, cache, table, lengths = made(msda, 11, dtype, fmt, B, S, N, D, page, [min(S, n) for n in lengths])
    q = normal(g, (B, T, M, D), C.DT[dtype])
    key, value = normal(g, (B, T, N, D), C.DT[dtype]), normal(g, (B, T, N, D), C.DT[dtype])
    if new == "none":
        compare(msda, q, cache, table, lengths)
    elif new == "chain":
        compare(msda, q, cache, table, lengths, key, value)
    elif new == "tree":
        compare(msda, q, cache, table, lengths, key, value, mask=tree(g, B, T))
    else:                                           # padding holds NaN
        counts = torch.randint(0, T + 1, (B,), generator=g, device=DEV).int()
        counts[0] = T
        behind = torch.arange(T, device=DEV)[None] >= counts[:, None]
        for x in (q, key, value):
            x[behind] = math.nan
        mask = (torch.rand((1, T, T), generator=g, device=DEV) < 0.6) if T > 1 else None
        compare(msda, q, cache, table, lengths, key, value, mask=mask, counts=counts)


MANY = [  # more rows a key head: heads that do not divide a tile of 128, one row more than a tile, several tiles
    (1, 33, 300, 1, 1, 16, 16), (2, 11, 1000, 12, 4, 80, 32), (1, 43, 700, 6, 2, 64, 64), (1, 300, 513, 2, 1, 128, 128),
    (3, 20, 2500, 16, 1, 48, 16), (1, 2, 900, 64, 1, 64, 16), (1, 1, 900, 100, 1, 128, 64), (1, 1, 600, 130, 1, 32, 16),
    (2, 64, 5000, 8, 2, 128, 256), (37, 18, 150, 1, 1, 32, 16), (9, 40, 200, 8, 8, 32, 32), (1, 129, 129, 4, 4, 112, 1024), (2, 260, 0, 2, 2, 64, 16),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("new", ["none", "chain", "tree", "ragged"])
@pytest.mark.parametrize("size", MANY, ids=lambda s: "x".join(map(str, s)))
def test_many_rows(msda, size, new, fmt, dtype):  # noqa: F811
    test_sizes(msda, size, new, fmt, dtype)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 20, 64])
def test_long_shares(msda, T, fmt, D):  # noqa: F811
    """Blocks that walk many tiles over the ends of several sequences, whose last tiles hold rows that are not theirs (NaN)."""
    lengths = [11999, 9000, 12001, 130, 7777, 10113, 5, 11000, 8191, 6401]
    g, cache, table, lengths = made(msda, 24, "bf16", fmt, 10, 12001, 4, D, 64, lengths)
    q, key, value = (normal(g, (10, T, n, D), torch.bfloat16) for n in (16, 4, 4))
    counts = torch.randint(1, T + 1, (10,), generator=g, device=DEV).int()
    for x in (q, key, value):
        x[torch.arange(T, device=DEV)[None] >= counts[:, None]] = math.nan
    for _ in range(2):
        compare(msda, q, cache, table, lengths, key, value, counts=counts)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T", [3, 60])
def test_rows_that_see_nothing(msda, fmt, dtype, T):  # noqa: F811
    g, cache, table, lengths = made(msda, 12, dtype, fmt, 3, 500, 2, 64, 32, [0, 500, 1])
    q, key, value = (normal(g, (3, T, n, 64), C.DT[dtype]) for n in (4, 2, 2))
    mask = torch.zeros((3, T, T), dtype=torch.bool, device=DEV)
    mask[0, 1, 0] = True
    out, lse = compare(msda, q, cache, table, lengths, key, value, mask=mask)
    assert not out[0, 0].any() and (lse[0, :, 0] == -math.inf).all() and lse[0, :, 1].isfinite().all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T", [1, 40])
def test_scores_that_rise_and_scales_far_apart(msda, fmt, dtype, T):  # noqa: F811
    """Keys whose scores grow along the sequence (the reference follows), values whose scales differ by 2^20."""
    B, S, N, D, page = 2, 3000, 2, 64, 64
    g, cache, table, lengths = made(msda, 13, dtype, fmt, B, S, N, D, page)
    q = normal(g, (B, T, 4, D), C.DT[dtype]).abs()
    k = normal(g, (B, S, N, D)) * 0.2 + torch.linspace(-2, 2, S, device=DEV)[None, :, None, None]
    v = normal(g, (B, S, N, D)) * torch.exp2(torch.randint(-10, 11, (B, S, N, 1), generator=g, device=DEV).float())
    msda.cache_write(cache, k.to(q.dtype), v.to(q.dtype), table, ints(0, 0))
    compare(msda, q, cache, table, lengths)
    msda.cache_write(cache, k.flip(1).to(q.dtype), v.to(q.dtype), table, ints(0, 0))
    compare(msda, q, cache, table, lengths, scale=0.7)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 40])
def test_values_without_an_order(msda, fmt, T):  # noqa: F811
    g, cache, table, lengths = made(msda, 14, "bf16", fmt, 2, 700, 2, 32, 16)
    q = normal(g, (2, T, 4, 32), torch.bfloat16)
    k = normal(g, (2, 700, 2, 32), torch.bfloat16)
    v = k.clone()
    v[0, 333, 0, 5] = math.nan
    k[1, 100, 1, 0] = math.nan
    msda.cache_write(cache, k, v, table, ints(0, 0))
    out, lse = msda.cache_attention(q, cache, table, lengths)
    out = out.view(2, T, 4, 32)
    assert out[0, :, :2, 5].isnan().all() and out[0, :, 2:].isfinite().all() and lse[0].isfinite().all()
    assert out[1, :, 2:].isnan().all() and lse[1, 2:].isnan().all() and out[1, :, :2].isfinite().all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 40])
def test_bad_pages_and_lengths(msda, fmt, T):  # noqa: F811
    """A token of a page that does not exist is not seen, a length beyond the table is the table's."""
    g, cache, table, lengths = made(msda, 15, "f16", fmt, 2, 640, 2, 64, 16)
    q = normal(g, (2, T, 4, 64), torch.float16)
    assert msda.device_errors() == 0
    bad = table.clone()
    bad[0, 3], bad[0, 20], bad[1, 39] = -1, 1 << 20, cache.key.shape[0]
    out, lse = msda.cache_attention(q, cache, bad, lengths)
    assert msda.device_errors() == 8
    keep = torch.ones(2, 640, dtype=torch.bool, device=DEV)
    keep[0, 48:64] = keep[0, 320:336] = keep[1, 624:] = False
    short = msda.cache_create(90, 16, 2, 64, C.FORMAT.get(fmt, torch.float16))
    k, v = (torch.zeros((2, 640, 2, 64), device=DEV, dtype=torch.float16) for _ in range(2))
    full = msda.cache_read(cache, table, lengths, 640, dtype=torch.float16)
    n = keep.sum(1).int()
    for b in range(2):
        k[b, :n[b]], v[b, :n[b]] = full[0][b, keep[b]], full[1][b, keep[b]]
    t2 = torch.arange(80, device=DEV).view(2, 40).int()
    msda.cache_write(short, k, v, t2, ints(0, 0))
    want = C.attention(q, short, t2, n)
    C.R.check(out, want["out"], "out")
    C.R.check(lse, want["lse"], "lse")
    far = msda.cache_attention(q, cache, table, ints(5000, -3))
    assert msda.device_errors() == 8
    near = msda.cache_attention(q, cache, table, ints(640, 0))
    assert all(torch.equal(a, b) for a, b in zip(far, near)) and msda.device_errors() == 0
    assert not near[0][1].any()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 50])
def test_equal_bits_streams_and_graphs(msda, fmt, T):  # noqa: F811
    g, cache, table, lengths = made(msda, 16, "bf16", fmt, 5, 4000, 2, 64, 32, [4000, 1, 0, 3999, 77])
    q, key, value = (normal(g, (5, T, n, 64), torch.bfloat16) for n in (8, 2, 2))
    want = msda.cache_attention(q, cache, table, lengths, key, value)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(msda.cache_attention(q, cache, table, lengths, key, value), want))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        s.wait_stream(torch.cuda.default_stream())
        other = msda.cache_attention(q, cache, table, lengths, key, value)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, want))
    graph, counts = torch.cuda.CUDAGraph(), ints(0, 0, 0, 0, 1)
    with torch.cuda.graph(graph):
        msda.cache_write(cache, key, value, table, lengths, counts=counts)
        got = msda.cache_attention(q, cache, table, lengths, key, value)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # lengths and tokens are read when the graph runs
    lengths.copy_(ints(3000, 1, 0, 1999, 5))
    q.neg_()
    want = C.attention(q, cache, table, lengths, key, value)
    graph.replay()
    torch.cuda.synchronize()
    C.R.check(got[0], want["out"], "out")
    C.R.check(got[1], want["lse"], "lse")


def test_a_bound_on_the_lengths(msda):  # noqa: F811
    g, cache, table, lengths = made(msda, 17, "f16", "e4m3", 4, 5000, 2, 64, 64, [200, 100, 300, 0])
    q = normal(g, (4, 1, 4, 64), torch.float16)
    want = C.attention(q, cache, table, lengths)
    for longest in (300, 512, 4000, None):
        out, lse = msda.cache_attention(q, cache, table, lengths, longest=longest)
        C.R.check(out, want["out"], "out")
        C.R.check(lse, want["lse"], "lse")
    got = msda.cache_attention(q, cache, table, lengths, longest=150)   # beyond the bound: cut, and told
    assert msda.device_errors() == 8
    want = C.attention(q, cache, table, lengths.clamp(max=150))
    C.R.check(got[0], want["out"], "out")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_prompt_drafts_and_tokens_together(msda, fmt, dtype):  # noqa: F811
    """A prompt in two pieces, then drafted trees of which a path is kept, then single tokens: each step's output is that of
    attention over the sequence so far (its cached part as the cache holds it)."""
    B, M, N, D, page = 3, 8, 2, 64, 16
    g = gen(18)
    cache = msda.cache_create(60, page, N, D, C.FORMAT.get(fmt, C.DT[dtype]))
    poison(cache)
    table = table_of(g, B, 20, 60)
    lengths = ints(0, 0, 0)
    make = lambda T: [normal(g, (B, T, n, D), C.DT[dtype]) for n in (M, N, N)]   # noqa: E731
    for T, counts in ((70, ints(70, 33, 1)), (41, ints(41, 0, 40))):
        q, k, v = make(T)
        compare(msda, q, cache, table, lengths, k, v, counts=counts)
        msda.cache_write(cache, k, v, table, lengths, counts=counts)
        lengths = lengths + counts
    for _ in range(3):
        q, k, v = make(12)
        mask = tree(g, B, 12)
        compare(msda, q, cache, table, lengths, k, v, mask=mask)
        path = torch.stack([mask[b, 11] for b in range(B)])             # the last token's ancestors are kept
        kept = path.sum(1).int()
        select = path.int().argsort(dim=1, descending=True, stable=True).int()
        msda.cache_write(cache, k, v, table, lengths, counts=kept, select=select)
        for b in range(B):
            n = int(kept[b])
            back = C.tokens(cache, table, b, int(lengths[b]) + n)[0][-n:]
            mine = k[b, select[b, :n].long()]
            want = mine.double() if fmt == "same" else C.stands_for(C.quantise(mine, C.FORMAT[fmt])[0].float(), C.quantise(mine, C.FORMAT[fmt])[1].to(torch.uint8))
            assert torch.equal(back, want)
        lengths = lengths + kept
        q, k, v = make(1)
        compare(msda, q, cache, table, lengths, k, v)
        msda.cache_write(cache, k, v, table, lengths)
        lengths = lengths + 1


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 40])
def test_padding_without_new_keys(msda, fmt, T):  # noqa: F811
    """counts alone: padded queries, NaN in them, over the cache."""
    g, cache, table, lengths = made(msda, 21, "f16", fmt, 3, 300, 2, 48, 32, [300, 0, 17])
    q = normal(g, (3, T, 4, 48), torch.float16)
    counts = ints(T, T, 0)
    q[2] = math.nan
    out, lse = compare(msda, q, cache, table, lengths, counts=counts)
    assert not out[1:].any() and (lse[1:] == -math.inf).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_two_calls_at_once(msda, fmt):  # noqa: F811
    """Calls on two streams over one cache, each with parts to join: the results of one after the other."""
    g, cache, table, lengths = made(msda, 22, "bf16", fmt, 2, 9000, 2, 128, 64)
    q = [normal(g, (2, T, 8, 128), torch.bfloat16) for T in (1, 40)]
    want = [msda.cache_attention(x, cache, table, lengths) for x in q]
    streams = [torch.cuda.Stream() for _ in q]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, x in zip(streams, q):
            with torch.cuda.stream(s):
                got.append(msda.cache_attention(x, cache, table, lengths))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_a_workspace_of_ones_own(msda):  # noqa: F811
    g, cache, table, lengths = made(msda, 23, "bf16", "int8", 2, 9000, 2, 64, 64)
    q = normal(g, (2, 3, 8, 64), torch.bfloat16)
    want = msda.cache_attention(q, cache, table, lengths)
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device=DEV)
    for _ in range(2):
        got = msda.cache_attention(q, cache, table, lengths, workspace=ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_against_dense_attention(msda):  # noqa: F811
    """A full prompt over an empty cache is causal attention; over rows in the cache it is its last rows."""
    g, cache, table, lengths = made(msda, 19, "bf16", "same", 2, 512, 4, 64, 32)
    q, k, v = (normal(g, (2, 700, n, 64), torch.bfloat16) for n in (8, 4, 4))
    want = msda.attention_forward(q, k, v, causal=True)
    msda.cache_write(cache, k[:, :512], v[:, :512], table, ints(0, 0))
    got = msda.cache_attention(q[:, 512:], cache, table, lengths, k[:, 512:], v[:, 512:])
    assert (got[0].float() - want[0][:, 512:].float()).norm() <= 4 * 2.0 ** -8 * want[0][:, 512:].float().norm()
    assert (got[1] - want[1][:, :, 512:]).abs().max() < 1e-4


def test_refusals(msda):  # noqa: F811
    g, cache, table, lengths = made(msda, 20, "bf16", "e4m3", 2, 100, 2, 32, 16)
    q, k, v = (normal(g, (2, 3, n, 32), torch.bfloat16) for n in (4, 2, 2))
    call = lambda *a, **kw: msda.cache_attention(*a, **kw)               # noqa: E731
    bad = [
        (ValueError, "heads", (q[:, :, :3], cache, table, lengths), {}),
        (ValueError, "channels", (q[..., :16], cache, table, lengths), {}),
        (TypeError, "int32", (q, cache, table.long(), lengths), {}),
        (TypeError, "int32", (q, cache, table, lengths.long()), {}),
        (ValueError, "lengths", (q, cache, table, lengths[:1]), {}),
        (ValueError, "table", (q, cache, table[:1], lengths), {}),
        (TypeError, "together", (q, cache, table, lengths, k), {}),
        (ValueError, "mask", (q, cache, table, lengths), {"mask": torch.ones(3, 3, dtype=torch.bool, device=DEV)}),
        (ValueError, "mask", (q, cache, table, lengths, k, v), {"mask": torch.ones(3, 4, dtype=torch.bool, device=DEV)}),
        (TypeError, "bool", (q, cache, table, lengths, k, v), {"mask": torch.ones(3, 3, device=DEV)}),
        (TypeError, "key is", (q, cache, table, lengths, k.half(), v), {}),
        (ValueError, "counts", (q, cache, table, lengths), {"counts": ints(1)}),
        (ValueError, "key_scale", (q, cache._replace(key_scale=None), table, lengths), {}),
        (ValueError, "cache.value", (q, cache._replace(value=cache.value[1:]), table, lengths), {}),
        (ValueError, "scales", (q, msda.cache_create(4, 16, 2, 32)._replace(key_scale=cache.key_scale), table, lengths), {}),
        (TypeError, "cache", (q.half(), msda.cache_create(9, 16, 2, 32), table, lengths), {}),
        (TypeError, "unsupported", (q.double(), cache, table, lengths), {}),
        (msda.MsdaError, "longest", (q, cache, table, lengths), {"longest": 113}),
        (msda.MsdaError, "longest", (q, cache, table, lengths), {"longest": -1}),
        (msda.MsdaError, "scale", (q, cache, table, lengths), {"scale": 0.0}),
        (msda.MsdaError, "workspace", (q, msda.cache_create(400, 16, 2, 32), torch.zeros((2, 200), dtype=torch.int32, device=DEV), lengths),
         {"workspace": torch.empty(16, dtype=torch.uint8, device=DEV)}),
        (ValueError, "workspace", (q, cache, table, lengths), {"workspace": torch.empty(1 << 20, dtype=torch.uint8)}),
        (ValueError, "no gradient", (q.clone().requires_grad_(), cache, table, lengths), {}),
    ]
    for kind, text, args, kw in bad:
        with pytest.raises(kind, match=text):
            call(*args, **kw)
    with torch.no_grad():
        call(q.clone().requires_grad_(), cache, table, lengths)
    write = lambda *a, **kw: msda.cache_write(cache, *a, **kw)           # noqa: E731
    for kind, text, args, kw in [
        (ValueError, "heads", (k[:, :, :1], v, table, lengths), {}),
        (ValueError, "value", (k, v[:, :2], table, lengths), {}),
        (ValueError, "start", (k, v, table, lengths[:1]), {}),
        (ValueError, "select", (k, v, table, lengths), {"select": ints(1, 2)}),
        (TypeError, "int32", (k, v, table, lengths), {"counts": lengths.long()}),
        (ValueError, "no gradient", (k.clone().requires_grad_(), v, table, lengths), {}),
    ]:
        with pytest.raises(kind, match=text):
            write(*args, **kw)
    with pytest.raises(TypeError, match="cache"):
        msda.cache_read(msda.cache_create(4, 16, 2, 32), table, lengths, 10, dtype=torch.float32)
    with pytest.raises(ValueError, match="lengths"):
        msda.cache_read(cache, table, ints(1, 2, 3), 10)
