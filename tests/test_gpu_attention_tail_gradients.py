"""Gradients of values that every query gives a small share, in binary16."""
import math

import pytest

import dense_reference as R
from test_gpu_attention import DEV, both, msda  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [32, 128])
@pytest.mark.parametrize("gap", [17.5, 19.3125, 19.40625])
def test_value_gradients_of_small_shares(msda, gap, D):  # noqa: F811
    """One key takes all but exp(-gap) a key, the same share for each query, so that the shares' roundings do not cancel: a share
    down to 2^-28 is rounded by 2^-11 of it, the result once more; scores, exponentials and the sum of 1000 in binary32 are off
    by less than 2^-12."""
    Q, S, M = 1000, 1100, 2
    q, k = torch.zeros(1, Q, M, D, device=DEV).half(), torch.zeros(1, S, M, D, device=DEV).half()
    q[..., 0], k[:, 0, :, 0] = 1, gap
    v = torch.zeros_like(k)
    do = torch.full((1, Q, M * D), 256.0, device=DEV).half()
    got = both(msda, q, k, v, do, {"scale": 1.0})
    share = math.exp(-gap) / (1 + (S - 1) * math.exp(-gap))
    want = Q * 256 * share
    assert float((got["grad_value"][:, 1:].double() / want - 1).abs().max()) <= 2 * 2.0 ** -11 + 2.0 ** -12


@pytest.mark.parametrize("size", [(3, 1, 5351, 2, 2, 72), (2, 1, 3000, 4, 4, 128)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("spread", [3, 6])
def test_key_gradients_of_one_query(msda, size, spread):  # noqa: F811
    """One query over a long axis, scores spread, gradients of a scaled loss: each key's gradient is one product of a small dS."""
    B, Q, S, M, N, D = size
    for seed in range(6):
        g = torch.Generator(device=DEV).manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g, device=DEV)   # noqa: E731
        q, k, v = (rnd(B, Q, M, D) * spread).half(), rnd(B, S, N, D).half(), rnd(B, S, N, D).half()
        do = (rnd(B, Q, M * D) * 300).half()
        want = R.attention(q, k, v, do)
        got = both(msda, q, k, v, do, {})
        for name in want:
            R.check(got[name], want[name], name)
