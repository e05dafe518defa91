"""Masks that empty whole tiles of queries and keys, other ones for each head."""
import pytest

import dense_reference as R
from test_gpu_attention import DEV, both, make, msda  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def band(kind, B, M, Q, S):
    i, j = torch.arange(Q, device=DEV)[:, None], torch.arange(S, device=DEV)[None]
    if kind == "band":                      # a row sees keys around its own place
        m = (i * S // Q - j).abs() < 50
    elif kind == "groups":                  # groups in front that see themselves and what follows; those only one another
        g = torch.where(torch.arange(max(Q, S), device=DEV) < 300, torch.arange(max(Q, S), device=DEV) // 75, -1)
        m = (g[None, :S] == -1) | (g[:Q, None] == g[None, :S])
    elif kind == "one corner":
        m = (i >= Q - 30) & (j < 40)
    else:                                   # each head and batch item a band of its own, the last head of the first item nothing
        at = torch.arange(B * M, device=DEV).view(B, M, 1, 1) * 97 % S
        m = (j - at - i // 3).abs() < 40
        m[0, -1] = False
    return m


@pytest.mark.parametrize("dtype,D", [("f32", 48), ("bf16", 64), ("f16", 128), ("bf16", 32), ("f32", 80)])
@pytest.mark.parametrize("kind", ["band", "groups", "one corner", "each"])
@pytest.mark.parametrize("more", ["", "keys", "causal"])
def test_tiles(msda, kind, more, dtype, D):  # noqa: F811
    B, Q, S, M, N = 2, 700, 650, 6, 2
    q, k, v, do = make(51, dtype, B, Q, S, M, N, D)
    m = band(kind, B, M, Q, S)
    kw, ok = {"mask": m}, m if m.dim() == 4 else m[None, None]
    if more == "keys":
        km = torch.arange(S, device=DEV)[None] < torch.tensor([[S], [S // 3]], device=DEV)
        kw["key_mask"], ok = km, ok & km[:, None, None]
    if more == "causal":
        kw["causal"] = True
        ok = ok & (torch.arange(S, device=DEV)[None] <= torch.arange(Q, device=DEV)[:, None] + (S - Q))[None, None]
    want = R.attention(q, k, v, do, ok)
    got = both(msda, q, k, v, do, kw)
    for name in want:
        R.check(got[name], want[name], name)


def test_many_rows(msda):  # noqa: F811
    """Two row tiles a block of the forward, each with other keys."""
    B, Q, S, M, N, D = 1, 5000, 1500, 8, 8, 32
    q, k, v, do = make(52, "bf16", B, Q, S, M, N, D)
    m = band("band", B, M, Q, S)
    want = R.attention(q, k, v, do, m[None, None])
    got = both(msda, q, k, v, do, {"mask": m})
    for name in want:
        R.check(got[name], want[name], name)
