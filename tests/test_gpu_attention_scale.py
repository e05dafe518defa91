"""The smallest scales that a call may give."""
import pytest

import dense_reference as R
from test_gpu_attention import both, make, masks, msda  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("f32", 80), ("f16", 64), ("bf16", 128), ("bf16", 20)])
@pytest.mark.parametrize("kind", ["keys none", "pairs", "causal"])
@pytest.mark.parametrize("scale", [1e-300, 1e-46, 1e-44, 1e-20])
def test_scales_that_binary32_hardly_holds(msda, scale, kind, dtype, D):  # noqa: F811
    """Scores are 0 to binary32: visible keys weigh the same, the others nothing."""
    B, Q, S, M, N = 2, 130, 300, 4, 2
    q, k, v, do = make(98, dtype, B, Q, S, M, N, D)
    kw, ok = masks(kind, 99, B, Q, S, M)
    want = R.attention(q, k, v, do, ok, scale=scale)
    got = both(msda, q, k, v, do, {**kw, "scale": scale})
    for name in want:
        R.check(got[name], want[name], name)
