"""Rows in which one key of the paged cache outweighs every other and the others still make the output."""
import pytest

import dense_reference as R
from test_gpu_cache import C, DEV, FORMATS, gen, ints, msda, table_of  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def tail(msda, fmt, dtype, B, T, S, M, N, D, gap, places, page=64):  # noqa: F811
    """Query t has a score of `gap` at key places[t % n] and 0 elsewhere; values are 0 at those keys, else 1."""
    n = len(places)
    q = torch.zeros(B, T, M, D, device=DEV)
    k = torch.zeros(B, S, N, D, device=DEV)
    v = torch.ones(B, S, N, D, device=DEV)
    for i, at in enumerate(places):
        q[:, i::n, :, i] = 1
        k[:, at, :, i] = gap
        v[:, at] = 0
    width = -(-S // page)
    cache = msda.cache_create(B * width, page, N, D, C.FORMAT.get(fmt, C.DT[dtype]))
    table = table_of(gen(37), B, width, B * width)
    msda.cache_write(cache, k.to(C.DT[dtype]), v.to(C.DT[dtype]), table, ints(*[0] * B))
    return q.to(C.DT[dtype]), cache, table


def check(msda, q, cache, table, lengths, dtype, fmt):  # noqa: F811
    out, lse = msda.cache_attention(q, cache, table, lengths, scale=1.0)
    for b in range(q.shape[0]):
        k, v = C.tokens(cache, table, b, int(lengths[b]))
        want = R.attention(q[b:b + 1], k[None], v[None], scale=1.0)
        value, bound = want["out"]
        if dtype == "f16" or fmt != "same":
            # what is rounded next to a tile's or a step's largest score, whose P is 2^8: half of binary16's smallest step,
            # 2^-25, for at most 127 keys
            bound = bound + 127 * 2.0 ** -33
        R.check(out[b:b + 1], (value, bound), "out")
        R.check(lse[b:b + 1], want["lse"], "lse")


# (B, T, S, M, N, D): one token, shared heads, more rows than a tile of 16, one and two tiles of 128, both widths
SIZES = [(1, 1, 22223, 8, 2, 64), (2, 3, 9000, 4, 4, 32), (1, 40, 22223, 2, 2, 64), (1, 30, 12000, 16, 2, 96), (2, 300, 5000, 4, 4, 64)]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("gap", [8.0, 14.0, 17.0, 17.625, 20.0, 25.0])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_dominant_key_over_a_heavy_tail(msda, size, gap, fmt, dtype):  # noqa: F811
    """Keys in the first, a middle and the last tile outweigh the rest by up to 7e10 each."""
    B, T, S, M, N, D = size
    q, cache, table = tail(msda, fmt, dtype, *size, gap, [0, S // 2, S - 1])
    check(msda, q, cache, table, ints(*[S] * B), dtype, fmt)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 40])
def test_whole_sequences_a_block(msda, T, fmt, dtype):  # noqa: F811
    """So many sequences that a block walks them whole, the outweighing key in its first, a middle or its last tile."""
    B, S, M, N, D = 60, 2600, 8, 8, 32
    q, cache, table = tail(msda, fmt, dtype, B, T, S, M, N, D, 18.0, [5, S // 2 + 1, S - 3])
    lengths = torch.where(torch.arange(B, device=DEV) % 3 == 0, S, S - 400).int()
    check(msda, q, cache, table, lengths, dtype, fmt)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 40])
def test_scores_that_fall_and_rise(msda, T, fmt, dtype):  # noqa: F811
    """Tiles whose scores fall by 13, then rise by 11 again and again: each needs another reference."""
    B, S, M, N, D, page = 2, 4000, 4, 4, 64, 32
    g = gen(38)
    q, k = torch.zeros(B, T, M, D, device=DEV), torch.zeros(B, S, N, D, device=DEV)
    v = torch.randn((B, S, N, D), generator=g, device=DEV)
    q[..., 0] = 1
    t = torch.arange(S, device=DEV) // 128
    k[..., 0] = torch.where(t % 2 == 0, 30.0 - t, 17.0 - t)[None, :, None]
    cache = msda.cache_create(260, page, N, D, C.FORMAT.get(fmt, C.DT[dtype]))
    table = table_of(g, B, 125, 260)
    msda.cache_write(cache, k.to(C.DT[dtype]), v.to(C.DT[dtype]), table, ints(0, 0))
    check(msda, q.to(C.DT[dtype]), cache, table, ints(S, 1999), dtype, fmt)
