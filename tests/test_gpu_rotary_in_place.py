"""Outputs that are their own inputs, through the C ABI."""
import pytest

from test_gpu_rotary import DEV, EPS, how, make, msda  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("size", [(2, 37, 3, 1, 32), (1, 300, 8, 2, 128), (2, 50, 4, 1, 96), (1, 65, 5, 2, 20), (1, 9, 3, 3, 7)],
                         ids=lambda s: "x".join(map(str, s)))
def test_in_place(msda, size, interleaved, dtype):  # noqa: F811
    """The bits of a call with outputs of its own."""
    from scale_deformable_attention_gb300 import _lib
    from scale_deformable_attention_gb300._rotary import _problem

    B, S, M, N, D = size
    q, k = make(75, dtype, B, S, (M, N), D)
    wq, wk = (1 + 0.2 * torch.randn((2, D), device=DEV, generator=torch.Generator(device=DEV).manual_seed(76))).to(q.dtype)
    h = how("float", B, S, (D // 4, D // 4 - D // 8))
    want = msda.norm_rotary_forward(q, k, wq, wk, *h, eps=EPS, interleaved=interleaved)
    alone = msda.rotary_forward(q, *h, interleaved=interleaved)
    lib, dt, st = _lib.lib(), {"f32": 0, "f16": 1, "bf16": 2}[dtype], torch.cuda.current_stream().cuda_stream
    flags = _lib.ROTARY_INTERLEAVED if interleaved else 0
    x, y = q.clone(), k.clone()
    _, _, pos, freq, p = _problem(x, y, *h)
    _lib.check(lib.msda_norm_rotary_forward(dt, flags, p, EPS, pos.data_ptr(), freq.data_ptr(), x.data_ptr(), y.data_ptr(),
                                            wq.data_ptr(), wk.data_ptr(), x.data_ptr(), y.data_ptr(), st))
    assert torch.equal(x, want[0]) and torch.equal(y, want[1])
    x = q.clone()
    _, _, pos, freq, p = _problem(x, None, *h)
    _lib.check(lib.msda_norm_rotary_forward(dt, flags, p, 0.0, pos.data_ptr(), freq.data_ptr(), x.data_ptr(), None, None, None,
                                            x.data_ptr(), None, st))
    assert torch.equal(x, alone)
