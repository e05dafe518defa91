"""Sums over long sequences in binary32 over a quantised cache: rounded to nearest, not cut off a little at each step."""
import pytest

from test_gpu_cache import C, DEV, gen, ints, msda, normal, table_of  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_positive_values(msda, fmt):  # noqa: F811
    """480 units, as many as there are blocks or more: each walks whole sequences, a warp 1050 groups of 16 keys.

    Adding 1050 groups, each rounded to nearest: at most half a step of the sum, 2^-24 of it, and as often up as down, so
    six standard deviations are 6 * sqrt(1050 / 3) * 2^-24 = 112 * 2^-24; the same for the sum of the probabilities, whose
    terms are as many steps of 32.  A probability is off by 2^-22 of it, a score (at most 0.1) by less, both at random over
    67200 keys.  2^-16 holds both; sums cut off downwards are off by 1050 to 2100 half steps, 2^-13.5 and more.
    """
    B, S, N, D, page = 15, 67200, 32, 16, 128
    g = gen(32)
    width = S // page
    cache = msda.cache_create(B * width, page, N, D, C.FORMAT[fmt])
    table = table_of(g, B, width, B * width)
    piece = 8400
    for at in range(0, S, piece):
        k = normal(g, (B, piece, N, D)) * 0.02
        v = 1 + torch.rand((B, piece, N, D), generator=g, device=DEV)
        msda.cache_write(cache, k, v, table, ints(*[at] * B))
    lengths = ints(*[S - 17 * b for b in range(B)])
    q = normal(g, (B, 1, N, D))
    out, lse = msda.cache_attention(q, cache, table, lengths)
    for b in range(B):
        k, v = C.tokens(cache, table, b, int(lengths[b]))
        s = torch.einsum("nd,knd->nk", q[b, 0].double(), k) / D ** 0.5
        want = torch.einsum("nk,knd->nd", s.softmax(-1), v)
        off = (out[b, 0].view(N, D).double() - want) / want
        assert off.abs().max() <= 2.0 ** -16
        assert (lse[b, :, 0].double() - s.logsumexp(-1)).abs().max() <= 2.0 ** -16
