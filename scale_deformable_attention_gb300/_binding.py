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
