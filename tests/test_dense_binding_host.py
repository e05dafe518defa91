"""The binding's own checks of the dense operators' arguments, on the host."""
import pytest

torch = pytest.importorskip("torch")


def test_workspace_lies_on_the_tensors_device_in_one_piece():
    from scale_deformable_attention_gb300._binding import workspace_of

    cpu, meta = torch.device("cpu"), torch.device("meta")
    buf = torch.empty(64, dtype=torch.uint8)
    assert workspace_of(64, buf, cpu) == (buf, 64)
    assert workspace_of(16, torch.empty((4, 4), dtype=torch.float32), cpu)[1] == 64
    assert workspace_of(0, None, cpu) == (None, 0)
    new, n = workspace_of(48, None, cpu)
    assert n == 48 and new.numel() == 48 and new.device == cpu
    with pytest.raises(ValueError, match="workspace"):
        workspace_of(16, buf, meta)
    with pytest.raises(ValueError, match="contiguous"):
        workspace_of(16, buf[::2], cpu)
    with pytest.raises(ValueError, match="contiguous"):
        workspace_of(16, torch.empty((8, 8), dtype=torch.uint8).t()[:, :4], cpu)


def test_positions_that_would_want_a_gradient():
    """Refused where a gradient would be recorded, taken under no_grad."""
    from scale_deformable_attention_gb300._rotary import _no_gradient

    plain, leaf = torch.ones(2), torch.ones(2, requires_grad=True)
    _no_gradient(plain, plain)
    for args in ((leaf, plain), (plain, leaf)):
        with pytest.raises(ValueError, match="detach"):
            _no_gradient(*args)
        with torch.no_grad():
            _no_gradient(*args)
