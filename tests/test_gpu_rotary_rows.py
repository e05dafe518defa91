"""Weights' gradients of the norm with rotation where a warp holds fewer rows than it has room for, without and with eps."""
import pytest

import dense_reference as R
from test_gpu_rotary import DEV, how, make, msda  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def check(msda, q, k, gq, gk, eps, interleaved, h):  # noqa: F811
    D = q.shape[3]
    wq, wk = (1 + 0.2 * torch.randn((2, D), device=DEV, generator=torch.Generator(device=DEV).manual_seed(72))).to(q.dtype)
    got = msda.norm_rotary_backward(q, k, wq, wk, *h, gq, gk, eps=eps, interleaved=interleaved)
    oq, ok = msda.norm_rotary_forward(q, k, wq, wk, *h, eps=eps, interleaved=interleaved)
    for x, w, g, out, dx, dw in ((q, wq, gq, oq, got[0], got[2]), (k, wk, gk, ok, got[1], got[3])):
        want = R.norm_rotary(x, w, *h, interleaved, eps, g)
        R.check(out, want["out"], "out")
        R.check(dx, want["grad"], "grad")
        R.check(dw, want["grad_weight"], "grad_weight")


# odd heads and a key head alone (two rows are worked on at once); tokens that leave part of a warp without one
SIZES = [(1, 1, 1, 1, 32), (2, 37, 3, 1, 32), (1, 131, 5, 1, 64), (3, 11, 8, 3, 128), (1, 7, 1, 1, 24), (2, 9, 3, 1, 20)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_no_eps(msda, size, interleaved, dtype):  # noqa: F811
    """eps = 0 is a norm like any other where no row is zero; rows that do not exist have no part in it."""
    B, S, M, N, D = size
    q, k, gq, gk = make(71, dtype, B, S, (M, N, M, N), D)
    check(msda, q, k, gq, gk, 0.0, interleaved, how("float", B, S, (D // 8, D // 8)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D", [32, 20])
def test_rows_of_zeros(msda, D, interleaved, dtype):  # noqa: F811
    """A row of zeros has the norm of eps alone: its gradient is w dz / sqrt(eps), the weights get none of it."""
    B, S, M, N = 2, 37, 3, 1
    q, k, gq, gk = make(73, dtype, B, S, (M, N, M, N), D)
    q[:, 3], k[:, 5] = 0, 0
    check(msda, q, k, gq, gk, 1e-4, interleaved, how("float", B, S, (D // 8, D // 8)))
