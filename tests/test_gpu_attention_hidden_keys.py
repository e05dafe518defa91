"""Keys that a mask leaves to some queries from which the causal order hides them: no query sees them."""
import math

import pytest

import dense_reference as R
from test_gpu_attention import DEV, both, make, msda  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,D", [("f32", 48), ("f32", 80), ("f16", 64), ("bf16", 128), ("bf16", 20)])
@pytest.mark.parametrize("Q,S", [(5, 6), (130, 300), (300, 130), (3, 1200)])
@pytest.mark.parametrize("each", [False, True])
def test_what_mask_and_order_hide_may_hold_anything(msda, each, Q, S, dtype, D):  # noqa: F811
    """A mask that shows most keys to the earlier half of the queries alone; what is hidden from all holds NaN and infinity."""
    B, M, N = 2, 4, 2
    q, k, v, do = make(101, dtype, B, Q, S, M, N, D)
    g = torch.Generator(device=DEV).manual_seed(102)
    mask = torch.rand((B, M, Q, S) if each else (Q, S), generator=g, device=DEV) < 0.6
    late = torch.rand((S,), generator=g, device=DEV) < 0.8
    mask[..., Q // 2:, :] &= ~late
    i, j = torch.arange(Q, device=DEV)[:, None], torch.arange(S, device=DEV)[None]
    ok = ((mask if each else mask[None, None]) & (j <= i + S - Q)).expand(B, M, Q, S)
    want = R.attention(q, k, v, do, ok)
    seen = ok.reshape(B, N, M // N, Q, S).any(3).any(2).transpose(1, 2)[..., None]
    assert not seen.all()
    empty = ~ok.any(-1).transpose(1, 2)[..., None]
    bad = torch.where(torch.arange(S, device=DEV) % 2 == 0, math.nan, math.inf)[None, :, None, None].to(k.dtype)
    k, v = torch.where(seen, k, bad), torch.where(seen, v, bad)
    q = torch.where(empty, torch.full_like(q, math.nan), q)
    do = torch.where(empty, torch.full_like(q, math.inf), do.view(B, Q, M, D)).reshape(B, Q, M * D)
    got = both(msda, q, k, v, do, {"mask": mask, "causal": True})
    for name in want:
        R.check(got[name], want[name], name)
