"""Rows in which one key outweighs every other and the others still make the output."""
import math

import pytest

import dense_reference as R
from test_gpu_attention import DEV, DT, make, masks, msda  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def tail(dtype, B, Q, S, M, N, D, gap, places, noise=0.0):
    """Row r has a score of gap[r % n] at key places[r % n] and about 0 elsewhere; values are 0 at those keys, else 1."""
    n = len(places)
    g = torch.Generator(device=DEV).manual_seed(81)
    q = torch.zeros(B, Q, M, D, device=DEV)
    k = noise * torch.randn(B, S, N, D, generator=g, device=DEV)
    v = torch.ones(B, S, N, D, device=DEV)
    for i, at in enumerate(places):
        q[:, i::n, :, i] = 1
        k[:, at, :, :] = 0
        k[:, at, :, i] = gap[i % len(gap)]
        v[:, at] = 0
    return q.to(DT[dtype]), k.to(DT[dtype]), v.to(DT[dtype])


# (B, Q, S, M, N, D): one and two row tiles a block, a split axis, both widths, shared heads
SIZES = [(1, 8, 22223, 2, 2, 32), (1, 300, 22223, 8, 8, 64), (2, 1000, 5000, 16, 16, 128), (1, 5, 20000, 8, 2, 96)]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("gap", [8.0, 14.0, 17.0, 17.625, 20.0, 25.0])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_dominant_key_over_a_heavy_tail(msda, size, gap, dtype):  # noqa: F811
    """Keys in the first, a middle and the last tile outweigh the rest by up to 7e10 each."""
    B, Q, S, M, N, D = size
    q, k, v = tail(dtype, *size, [gap], [0, S // 2, S - 1])
    want = R.attention(q, k, v, scale=1.0)
    out, lse = msda.attention_forward(q, k, v, scale=1.0)
    # what a tile holds beside its largest score is rounded to half of binary16's smallest step, 2^-25, where that score's P is
    # 2^8: 2^-33 of it, for at most 127 keys of the one tile against the tail of all S, exp(-gap) a key
    value, bound = want["out"]
    if dtype == "f16":
        bound = bound + 127 * 2.0 ** -33
    R.check(out, (value, bound), "out")
    R.check(lse, want["lse"], "lse")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("kind", ["keys", "pairs", "causal"])
def test_with_masks(msda, kind, dtype):  # noqa: F811
    """Masks that empty tiles between the dominant key and the tail, and rows that see the tail alone."""
    size = B, Q, S, M, N, D = 2, 400, 3000, 4, 4, 64
    q, k, v = tail(dtype, *size, [17.0, 19.5, 12.25], [1, 700, S - 2], 0.25)
    kw, ok = masks(kind, 82, B, Q, S, M)
    if "mask" in kw:
        kw["mask"][:, 128:1000] = False
    if "key_mask" in kw:
        kw["key_mask"][:, 128:640] = False
        kw["key_mask"][:, [1, 700, S - 2]] = True
    want = R.attention(q, k, v, None, ok, scale=1.0)
    out, lse = msda.attention_forward(q, k, v, scale=1.0, **kw)
    value, bound = want["out"]
    R.check(out, (value, bound + 127 * 2.0 ** -33 if dtype == "f16" else bound), "out")
    R.check(lse, want["lse"], "lse")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_scores_that_fall_and_rise(msda, dtype):  # noqa: F811
    """Tiles whose scores fall by 13, then rise by 11 again and again: each needs another reference."""
    B, Q, S, M, D = 1, 260, 4000, 8, 64
    q, k, v, _ = make(83, dtype, B, Q, S, M, M, D)
    q, k = torch.zeros_like(q), torch.zeros_like(k)
    q[..., 0] = 1
    t = torch.arange(S, device=DEV) // 128
    k[..., 0] = torch.where(t % 2 == 0, 30.0 - t, 17.0 - t)[None, :, None].to(k.dtype)
    want = R.attention(q, k, v, scale=1.0)
    out, lse = msda.attention_forward(q, k, v, scale=1.0)
    R.check(out, want["out"], "out")
    R.check(lse, want["lse"], "lse")


def test_two_levels_below(msda):  # noqa: F811
    """Three sizes of scores, values of the larger two cancelling: what is left is the smallest ones' share of 2^-30."""
    B, Q, S, M, D = 1, 140, 9000, 2, 32
    q, k, v, _ = make(84, "f16", B, Q, S, M, M, D)
    q, k, v = torch.zeros_like(q), torch.zeros_like(k), torch.full_like(v, 30000.0)
    q[..., 0] = 1
    k[:, 0, :, 0], v[:, 0] = 30.0, 0
    k[:, 1:300, :, 0], v[:, 1:300] = 15.0, 0
    want = R.attention(q, k, v, scale=1.0)
    out, lse = msda.attention_forward(q, k, v, scale=1.0)
    value, bound = want["out"]
    assert 0 < float(value.max()) < 2.0 ** -10
    R.check(out, (value, bound + 127 * 2.0 ** -33 * math.exp(-15) * 30000), "out")
    R.check(lse, want["lse"], "lse")
