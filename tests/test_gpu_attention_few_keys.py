"""Gradients of rows that see few keys of a long axis, in 16 bits."""
import pytest

import dense_reference as R
from test_gpu_attention import DEV, both, make, msda  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def few(kind, B, Q, S):
    if kind == "causal":
        i = torch.arange(Q, device=DEV)[:, None] + (S - Q)
        return {"causal": True}, (torch.arange(S, device=DEV)[None] <= i)[None, None]
    km = torch.zeros(B, S, dtype=torch.bool, device=DEV)
    km[0, 5] = km[1, S - 3:] = True
    return {"key_mask": km}, km[:, None, None]


@pytest.mark.parametrize("dtype,D", [("bf16", 32), ("f16", 64), ("bf16", 128), ("f16", 72)])
@pytest.mark.parametrize("kind", ["causal", "keys"])
def test_one_key_gives_no_gradient(msda, kind, dtype, D):  # noqa: F811
    """p = 1 at one key: dP - delta is zero, however long the axis is."""
    B, Q, S, M, N = 2, 400, 400, 4, 2
    q, k, v, do = make(41, dtype, B, Q, S, M, N, D)
    kw, _ = few(kind, B, Q, S)
    got = both(msda, q, k, v, do, kw)
    if kind == "causal":
        assert (got["grad_query"][:, 0] == 0).all()
    else:
        assert (got["grad_query"][0] == 0).all() and (got["grad_key"][0] == 0).all()


@pytest.mark.parametrize("D", [32, 128])
@pytest.mark.parametrize("kind", ["causal", "keys"])
def test_few_keys_of_many(msda, kind, D):  # noqa: F811
    """Left are the roundings of dS, of P and of the result, each uniform within 2^-8 (2^-8 / sqrt(3) of a value in the
    root mean square): at most 2^-8 together."""
    B, Q, S, M = 2, 500, 500, 16
    q, k, v, do = make(42, "bf16", B, Q, S, M, M, D)
    kw, ok = few(kind, B, Q, S)
    want = R.attention(q, k, v, do, ok)
    got = both(msda, q, k, v, do, kw)
    for name in ("grad_query", "grad_key", "grad_value"):
        value = want[name][0]
        assert float((got[name].double() - value).norm() / value.norm()) <= 2.0 ** -8, name
