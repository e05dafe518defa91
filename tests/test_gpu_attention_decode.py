"""Attention of a few query rows over a long key axis."""
import math

import pytest

import dense_reference as R
from test_gpu_attention import DEV, DT, make, masks, msda  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SIZES = [
    # B, Q, S, M, N, D
    (1, 1, 256, 1, 1, 8), (3, 1, 3001, 8, 2, 64), (2, 2, 1111, 8, 2, 128), (1, 8, 700, 3, 3, 32), (2, 3, 999, 4, 2, 24),
    (1, 1, 30000, 2, 2, 96), (4, 1, 257, 16, 2, 40), (40, 1, 300, 8, 8, 16), (1, 5, 2500, 1, 1, 112),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind", ["", "keys none", "pairs", "pairs each causal", "keys causal"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_sizes_and_masks(msda, size, kind, dtype):  # noqa: F811
    B, Q, S, M, N, D = size
    q, k, v, _ = make(61, dtype, *size)
    kw, ok = masks(kind, 62, B, Q, S, M)
    want = R.attention(q, k, v, None, ok)
    out, lse = msda.attention_forward(q, k, v, **kw)
    R.check(out, want["out"], "out")
    R.check(lse, want["lse"], "lse")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_cache_with_room(msda, dtype):  # noqa: F811
    """Keys and values in a cache [B, heads, room, 2, D] with more room than is filled, what lies behind being NaN."""
    B, Q, S, M, N, D = 2, 1, 1500, 8, 4, 64
    q, k, v, _ = make(63, dtype, B, Q, S, M, N, D)
    cache = torch.full((B, N, 2000, 2, D), math.nan, device=DEV, dtype=DT[dtype])
    cache[:, :, :S, 0], cache[:, :, :S, 1] = k.transpose(1, 2), v.transpose(1, 2)
    kc, vc = cache[:, :, :S, 0].transpose(1, 2), cache[:, :, :S, 1].transpose(1, 2)
    want, want_lse = msda.attention_forward(q, k, v)
    out, lse = msda.attention_forward(q, kc, vc)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    km = (torch.arange(2000, device=DEV) < S)[None]
    full = msda.attention_forward(q, cache[:, :, :, 0].transpose(1, 2), cache[:, :, :, 1].transpose(1, 2), key_mask=km)
    ref = R.attention(q, k, v)
    R.check(full[0], ref["out"], "out")
    R.check(full[1], ref["lse"], "lse")


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_values_without_an_order(msda, dtype):  # noqa: F811
    q, k, v, _ = make(64, dtype, 1, 2, 600, 4, 2, 32)
    q[0, 1, 2] = math.nan
    v[0, 77, 0, 3] = math.inf
    out, lse = msda.attention_forward(q, k, v)
    out = out.view(2, 4, 32)
    assert out[1, 2].isnan().all() and lse[0, 2, 1].isnan()
    assert (out[:, :2, 3] == math.inf).all()
    keep = torch.ones(2, 4, 32, dtype=torch.bool, device=DEV)
    keep[1, 2] = False
    keep[:, :2, 3] = False
    assert out[keep].isfinite().all()
    # hidden behind a mask both are nothing
    km = torch.ones(1, 600, dtype=torch.bool, device=DEV)
    km[0, 77] = False
    assert msda.attention_forward(q, k, v, key_mask=km)[0].view(2, 4, 32)[:, :2].isfinite().all()


def test_replayed_and_on_another_stream(msda):  # noqa: F811
    q, k, v, _ = make(65, "bf16", 2, 1, 5000, 8, 2, 64)
    want = msda.attention_forward(q, k, v)[0]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        s.wait_stream(torch.cuda.default_stream())
        other = msda.attention_forward(q, k, v)[0]
    torch.cuda.synchronize()
    assert torch.equal(other, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = msda.attention_forward(q, k, v)[0]
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
