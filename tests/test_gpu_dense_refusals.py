"""Workspaces that the dense operators refuse before any launch."""
import pytest

from test_gpu_attention import DEV, make, msda  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def workspaces():
    n = 64 << 20
    return torch.empty(n, dtype=torch.uint8), torch.empty(2 * n, dtype=torch.uint8, device=DEV)[::2]


def test_attention(msda):  # noqa: F811
    q, k, v, do = make(95, "f32", 1, 4, 3000, 4, 2, 32)
    out, lse = msda.attention_forward(q, k, v)
    for bad in workspaces():
        with pytest.raises(ValueError, match="workspace"):
            msda.attention_forward(q, k, v, workspace=bad)
        with pytest.raises(ValueError, match="workspace"):
            msda.attention_backward(q, k, v, out, lse, do, workspace=bad)


def test_norm_rotary(msda):  # noqa: F811
    q, k, _, _ = make(96, "bf16", 1, 5, 5, 4, 2, 32)
    w, pos, freq = torch.ones(32, device=DEV, dtype=q.dtype), torch.rand(1, 5, 1, device=DEV), torch.ones(16, device=DEV)
    for bad in workspaces():
        with pytest.raises(ValueError, match="workspace"):
            msda.norm_rotary_backward(q, k, w, w, pos, freq, (16,), q, k, workspace=bad)


def test_sampled_attention(msda):  # noqa: F811
    g = torch.Generator(device=DEV).manual_seed(97)
    rnd = lambda *s: torch.rand(s, generator=g, device=DEV)   # noqa: E731
    shapes = torch.tensor([[4, 5], [2, 3]], device=DEV)
    value, loc, attn, do = rnd(1, 26, 2, 32).half(), rnd(1, 7, 2, 2, 4, 2).half(), rnd(1, 7, 2, 2, 4).half(), rnd(1, 7, 64).half()
    for bad in workspaces():
        with pytest.raises(ValueError, match="workspace"):
            msda.backward(value, shapes, None, loc, attn, do, accum="fp32", workspace=bad)
