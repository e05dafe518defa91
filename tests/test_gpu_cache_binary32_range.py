"""binary32 values that bfloat16 does not hold, in an unquantised cache, in queries and in new tokens."""
import math

import pytest

from test_gpu_cache import C, msda, normal  # noqa: F401
from test_gpu_cache_attention import made

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("what", [math.inf, -math.inf, 3.4e38])
def test_above_the_largest(msda, what, T):  # noqa: F811
    """binary32 values above bf16's largest count as NaN, infinities among them: in a key every score of its head, in a value
    its channel, in a query its row.  Nothing else is touched."""
    g, cache, table, lengths = made(msda, 39, "f32", "same", 3, 300, 2, 32, 16)
    q = normal(g, (3, T, 4, 32))
    cache.key[table[0, 2].long(), 7, 1, 3] = what
    cache.value[table[1, 4].long(), 1, 0, 9] = what
    q[2, 0, 1, 5] = what
    out, lse = msda.cache_attention(q, cache, table, lengths)
    out = out.view(3, T, 4, 32)
    nan = torch.zeros_like(out, dtype=torch.bool)
    nan[0, :, 2:] = True
    nan[1, :, :2, 9] = True
    nan[2, 0, 1] = True
    assert torch.equal(out.isnan(), nan) and out[~nan].isfinite().all()
    nan = torch.zeros_like(lse, dtype=torch.bool)
    nan[0, 2:] = True
    nan[2, 1, 0] = True
    assert torch.equal(lse.isnan(), nan) and lse[~nan].isfinite().all()


@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("fmt", ["same", "int8"])
def test_new_tokens(msda, fmt, T):  # noqa: F811
    """The same for new tokens, over codes too: their products run as those of an unquantised cache."""
    g, cache, table, lengths = made(msda, 39, "f32", fmt, 3, 300, 2, 32, 16)
    q, k, v = (normal(g, (3, T, n, 32)) for n in (4, 2, 2))
    k[0, 0, 1, 3], v[1, 0, 0, 9] = math.inf, -math.inf          # seen by every query
    out, lse = msda.cache_attention(q, cache, table, lengths, k, v)
    out = out.view(3, T, 4, 32)
    nan = torch.zeros_like(out, dtype=torch.bool)
    nan[0, :, 2:] = True
    nan[1, :, :2, 9] = True
    assert torch.equal(out.isnan(), nan) and out[~nan].isfinite().all()
    assert lse[0, 2:].isnan().all() and lse[0, :2].isfinite().all() and lse[1:].isfinite().all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("fmt", ["same", "e4m3"])
@pytest.mark.parametrize("T", [5, 40])
def test_hidden_values(msda, T, fmt, dtype):  # noqa: F811
    """NaN in the value of a new token that no query sees: other sequences, heads and channels and every lse are as without it."""
    g, cache, table, lengths = made(msda, 43, dtype, fmt, 2, 300, 2, 32, 16)
    q, k, v = (normal(g, (2, T, n, 32), C.DT[dtype]) for n in (4, 2, 2))
    mask = torch.ones((2, T, T), dtype=torch.bool, device=q.device).tril()
    mask[0, :, 2] = False
    want = msda.cache_attention(q, cache, table, lengths, k, v, mask=mask)
    v[0, 2, 1, 7] = math.nan
    out, lse = msda.cache_attention(q, cache, table, lengths, k, v, mask=mask)
    same = torch.ones((2, T, 4, 32), dtype=torch.bool, device=q.device)
    same[0, :, 2:, 7] = False
    assert torch.equal(lse, want[1]) and torch.equal(out.view(2, T, 4, 32)[same], want[0].view(2, T, 4, 32)[same])
