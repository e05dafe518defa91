"""Strides, far pages and masks of every layout where a key head has more rows than the kernel of few rows takes."""
import pytest

from test_gpu_cache import C, DEV, FORMATS, gen, ints, msda, normal, table_of  # noqa: F401
from test_gpu_cache_attention import compare, made, tree

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T", [20, 150])
def test_slices_of_a_fused_projection(msda, T, dtype, fmt):  # noqa: F811
    """Queries, keys and values side by side in one tensor; sequences, then tokens, first in memory."""
    B, M, N, D = 2, 8, 4, 64
    g, cache, table, lengths = made(msda, 51, dtype, fmt, B, 400, N, D, 16, [400, 261])
    for shape, perm in (((B, T, M + 2 * N, D), (0, 1, 2, 3)), ((T, B, M + 2 * N, D), (1, 0, 2, 3)), ((B, M + 2 * N, T, D), (0, 2, 1, 3))):
        x = normal(g, shape, C.DT[dtype]).permute(perm)
        q, k, v = x.split((M, N, N), 2)
        compare(msda, q, cache, table, lengths, k, v)
        compare(msda, q, cache, table, lengths, k, v, mask=tree(g, B, T))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [48, 128])
def test_pools_of_any_layout(msda, D, fmt):  # noqa: F811
    """Token by token, K next to V in one pool, wider pages than their tokens: the same bits as head by head."""
    B, T, M, N, page, S = 2, 25, 8, 4, 32, 300
    g, plain, table, lengths = made(msda, 52, "bf16", fmt, B, S, N, D, page, [S, 177])
    n = plain.key.shape[0]
    both = torch.zeros((n, page + 16, 2, N, D), device=DEV, dtype=torch.uint8 if fmt != "same" else torch.bfloat16)
    both = both.view(plain.key.dtype)
    scales = torch.zeros((n, 2, page, N + 3), device=DEV, dtype=torch.uint8)
    cache = msda.PagedCache(both[:, :page, 0], both[:, 16:, 1], *((scales[:, 0, :, 1:N + 1], scales[:, 1, :, :N]) if fmt != "same" else ()))
    for a, b in zip(cache, plain):
        if a is not None:
            a.view(torch.uint8 if a.element_size() == 1 else torch.int16).copy_(b.view(torch.uint8 if b.element_size() == 1 else torch.int16))
    q, k, v = (normal(g, (B, T, h, D), torch.bfloat16) for h in (M, N, N))
    for args in ((), (k, v)):
        for a, b in zip(msda.cache_attention(q, cache, table, lengths, *args), compare(msda, q, plain, table, lengths, *args)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", ["same", "e4m3"])
def test_far_pages(msda, fmt):  # noqa: F811
    """Offsets beyond 32 bits: pages behind 2^32 elements, 80 rows a key head."""
    g = gen(53)
    pages, page, N, D = 135000, 256, 1, 128         # 4.4e9 elements
    cache = msda.cache_create(pages, page, N, D, C.FORMAT.get(fmt, torch.bfloat16))
    table = ints([pages - 1, 0], [pages - 2, pages // 2])
    key, value = normal(g, (2, 300, N, D), torch.bfloat16), normal(g, (2, 300, N, D), torch.bfloat16)
    msda.cache_write(cache, key, value, table, ints(0, 5))
    q = normal(g, (2, 20, 4, D), torch.bfloat16)
    compare(msda, q, cache, table, ints(300, 305))
    compare(msda, q, cache, table, ints(300, 200), key[:, :20], value[:, :20])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("which", ["query", "heads", "tokens", "new", "all"])
def test_broadcast_tensors(msda, which, fmt):  # noqa: F811
    """Strides of 0, which no tensor map takes."""
    B, T, M, N, D = 3, 30, 8, 2, 64
    g, cache, table, lengths = made(msda, 54, "f16", fmt, B, 500, N, D, 32, [500, 77, 0])
    q, k, v = (normal(g, (B, T, h, D), torch.float16) for h in (M, N, N))
    if which in ("query", "all"):
        q = q[:1].expand(B, T, M, D)
    if which == "heads":
        q = q[:, :, :1].expand(B, T, M, D)
    if which == "tokens":
        q = q[:, :1].expand(B, T, M, D)
    if which in ("new", "all"):
        k, v = k[:1].expand(B, T, N, D), v[:, :, :1].expand(B, T, N, D)
    compare(msda, q, cache, table, lengths, k, v)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", ["same", "int8"])
@pytest.mark.parametrize("T", [5, 33, 140])
def test_masks_of_any_layout(msda, T, fmt, dtype):  # noqa: F811
    """Two dimensions, one for all sequences, rows apart, rows that begin at any byte, keys that are not contiguous."""
    B, M, N, D = 2, 4, 2, 32
    g, cache, table, lengths = made(msda, 55, dtype, fmt, B, 200, N, D, 16, [200, 31])
    q, k, v = (normal(g, (B, T, h, D), C.DT[dtype]) for h in (M, N, N))
    big = torch.rand((B, T + 2, 2 * T + 3), generator=g, device=DEV) < 0.5
    for mask in (big[0, :T, :T], big[:1, 1:T + 1, 3:T + 3], big[:, 2:, 1:T + 1], big[:, :T, :2 * T:2], big[:, :T, :T].transpose(1, 2),
                 big[:1, :1, :T].expand(B, T, T)):
        compare(msda, q, cache, table, lengths, k, v, mask=mask)
        compare(msda, q, cache, table, lengths, k, v, mask=mask, counts=ints(T - 2, T))
