"""What the cache's operators refuse for want of a gradient, on the host."""
import pytest

torch = pytest.importorskip("torch")
import torch.autograd.forward_ad as fwAD  # noqa: E402


def test_reverse_and_forward_mode():
    from scale_deformable_attention_gb300._cache import _no_gradient

    plain, leaf = torch.ones(2), torch.ones(2, requires_grad=True)
    _no_gradient(plain, None, plain)
    with pytest.raises(ValueError, match="no gradient"):
        _no_gradient(plain, leaf)
    with torch.no_grad():
        _no_gradient(plain, leaf)
    with fwAD.dual_level():
        dual = fwAD.make_dual(plain, torch.ones(2))
        _no_gradient(plain, None)
        for args in ((dual,), (plain, dual), (None, dual)):
            with pytest.raises(ValueError, match="no gradient"):
                _no_gradient(*args)
            with torch.no_grad(), pytest.raises(ValueError, match="no gradient"):    # a tangent goes through no_grad
                _no_gradient(*args)
    _no_gradient(plain)
