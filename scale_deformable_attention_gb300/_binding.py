"""What the operators' bindings share: raw pointers, the current stream, the device."""
from __future__ import annotations

import contextlib
from typing import Optional

import torch

DTYPE_CODE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_HERE = contextlib.nullcontext()


def ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def stream(device: torch.device) -> int:
    """The current stream of ``device`` as a pointer (without the Stream object around it, which costs 2 us a call)."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def on_device(device: torch.device):
    """``device`` as the current one (nothing to switch where it is already)."""
    return _HERE if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def workspace_of(need: int, workspace: Optional[torch.Tensor], device: torch.device):
    """(workspace, its bytes) for a call that needs ``need``: the given one, checked, or a new one.  A kernel writes all
    bytes between its first and its last, so it lies on ``device`` in one piece."""
    if workspace is None:
        return (torch.empty(need, dtype=torch.uint8, device=device), need) if need else (None, 0)
    if workspace.device != device:
        raise ValueError(f"workspace is on {workspace.device}, the tensors on {device}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace, workspace.numel() * workspace.element_size()
