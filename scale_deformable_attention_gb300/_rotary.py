"""Rotary positions with several axes, alone and behind the norm of queries and
keys per head (C ABI ``msda_norm_rotary_forward`` / ``_backward``)."""
from __future__ import annotations

from typing import Optional, Sequence, Tuple

import torch

from . import _lib
from ._binding import DTYPE_CODE, on_device, ptr, stream, workspace_of

POSITION_CODE = {torch.float32: 0, torch.int32: 1, torch.int64: 2}


def _rows(name: str, x: torch.Tensor) -> torch.Tensor:
    """``x`` [B, S, heads, D] with its channels contiguous (a copy where they are not)."""
    if x.dim() != 4:
        raise ValueError(f"{name} must be [B, S, heads, D], got shape {tuple(x.shape)}")
    if x.dtype not in DTYPE_CODE:
        raise TypeError(f"{name}: unsupported dtype {x.dtype}; use float32, float16 or bfloat16")
    return x if x.stride(3) == 1 or x.shape[3] <= 1 else x.contiguous()


def _like(name: str, t: torch.Tensor, shape, x: torch.Tensor) -> torch.Tensor:
    if t is None:
        raise TypeError(f"{name} is missing")
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != x.dtype:
        raise TypeError(f"{name} is {t.dtype}, query {x.dtype}; all float tensors share one dtype")
    if t.device != x.device:
        raise ValueError(f"{name} is on {t.device}, query on {x.device}")
    return t.contiguous()


def _problem(query, key, positions, frequencies, sections):
    """Checks, and the C ABI's problem: (query, key, positions, frequencies, problem)."""
    query = _rows("query", query)
    B, S, M, D = query.shape
    dev = query.device
    if dev.type != "cuda":
        raise ValueError("the operator runs on CUDA tensors only (there is no CPU implementation)")
    N, ks = 0, (0, 0, 0)
    if key is not None:
        key = _rows("key", key)
        N = key.shape[2]
        if key.shape != (B, S, N, D):
            raise ValueError(f"key must be [B={B}, S={S}, heads, D={D}], got {tuple(key.shape)}")
        if key.dtype != query.dtype or key.device != dev:
            raise TypeError(f"key must be a {query.dtype} tensor on {dev}")
        ks = key.stride()
    sections = tuple(map(int, sections))
    A, P = len(sections), sum(sections)
    if not 1 <= A <= 4:
        raise ValueError(f"sections must name 1 to 4 axes, got {sections}")
    if positions.dtype not in POSITION_CODE:
        raise TypeError(f"positions must be float32, int32 or int64, got {positions.dtype}")
    if positions.shape not in ((B, S, A), (1, S, A)):
        raise ValueError(f"positions must be [{B} or 1, S={S}, {A}], got {tuple(positions.shape)}")
    if frequencies.shape != (P,) or frequencies.dtype != torch.float32:
        raise ValueError(f"frequencies must be a float32 tensor of the sections' sum {P}, "
                         f"got {frequencies.dtype} {tuple(frequencies.shape)}")
    if positions.device != dev:
        raise ValueError(f"positions is on {positions.device}, query on {dev}")
    if frequencies.device != dev:
        raise ValueError(f"frequencies is on {frequencies.device}, query on {dev}")
    positions = positions.contiguous()
    frequencies = frequencies.contiguous()
    qs = query.stride()
    p = _lib.RotaryProblem(B, S, M, N, D, A, *(sections + (0,) * (4 - A)), qs[0], qs[1], qs[2], ks[0], ks[1], ks[2],
                           POSITION_CODE[positions.dtype], S * A if positions.shape[0] > 1 else 0)
    return query, key, positions, frequencies, p


def _dense(x: torch.Tensor) -> torch.Tensor:
    return torch.empty_like(x) if x.is_contiguous() else torch.empty(x.shape, dtype=x.dtype, device=x.device)


def _forward(query, key, wq, wk, positions, frequencies, sections, eps, flags):
    query, key, positions, frequencies, p = _problem(query, key, positions, frequencies, sections)
    D = query.shape[3]
    if key is not None:
        wq = _like("query_weight", wq, (D,), query)
        wk = _like("key_weight", wk, (D,), query)
    q_out = _dense(query)
    k_out = None if key is None else _dense(key)
    with on_device(query.device):
        _lib.check(_lib.lib().msda_norm_rotary_forward(
            DTYPE_CODE[query.dtype], flags, p, eps, ptr(positions), ptr(frequencies), ptr(query), ptr(key), ptr(wq),
            ptr(wk), ptr(q_out), ptr(k_out), stream(query.device)))
    return q_out, k_out


def rotary_forward(x: torch.Tensor, positions: torch.Tensor, frequencies: torch.Tensor, sections: Sequence[int], *,
                   interleaved: bool = False) -> torch.Tensor:
    """``x`` [B, S, M, D] with its pairs of channels turned by position times
    frequency (C ABI ``msda_norm_rotary_forward`` without weights).

    ``positions`` [B or 1, S, axes]: float32, int32 or int64, one value an axis
    (time, height, width; or the x and y of a reference point).
    ``frequencies`` [sum(sections)] float32; ``sections[a]`` pairs turn by axis ``a``.
    Pairs are channels (j, j + sum(sections)), or (2j, 2j + 1) if ``interleaved``;
    channels behind them pass through.
    """
    return _forward(x, None, None, None, positions, frequencies, sections, 0.0,
                    _lib.ROTARY_INTERLEAVED if interleaved else 0)[0]


def rotary_backward(grad_out: torch.Tensor, positions: torch.Tensor, frequencies: torch.Tensor,
                    sections: Sequence[int], *, interleaved: bool = False) -> torch.Tensor:
    """Gradient of ``rotary_forward``'s input: the rotation by the negative angles."""
    return _forward(grad_out, None, None, None, positions, frequencies, sections, 0.0,
                    _lib.ROTARY_INVERSE | (_lib.ROTARY_INTERLEAVED if interleaved else 0))[0]


def norm_rotary_forward(query: torch.Tensor, key: torch.Tensor, query_weight: torch.Tensor, key_weight: torch.Tensor,
                        positions: torch.Tensor, frequencies: torch.Tensor, sections: Sequence[int], *,
                        eps: float = 1e-6, interleaved: bool = False) -> Tuple[torch.Tensor, torch.Tensor]:
    """Queries [B, S, M, D] and keys [B, S, N, D], each row normed over its D
    channels (x w / sqrt(mean(x^2) + eps)) and rotated as by ``rotary_forward``,
    in one pass (C ABI ``msda_norm_rotary_forward``).  Weights [D]."""
    if key is None:
        raise TypeError("key is missing")
    return _forward(query, key, query_weight, key_weight, positions, frequencies, sections, float(eps),
                    _lib.ROTARY_INTERLEAVED if interleaved else 0)


def norm_rotary_backward(query: torch.Tensor, key: torch.Tensor, query_weight: torch.Tensor, key_weight: torch.Tensor,
                         positions: torch.Tensor, frequencies: torch.Tensor, sections: Sequence[int],
                         grad_query_out: torch.Tensor, grad_key_out: torch.Tensor, *, eps: float = 1e-6,
                         interleaved: bool = False, workspace: Optional[torch.Tensor] = None
                         ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """(grad_query, grad_key, grad_query_weight, grad_key_weight) (C ABI ``msda_norm_rotary_backward``)."""
    if key is None:
        raise TypeError("key is missing")
    query, key, positions, frequencies, p = _problem(query, key, positions, frequencies, sections)
    D = query.shape[3]
    wq = _like("query_weight", query_weight, (D,), query)
    wk = _like("key_weight", key_weight, (D,), query)
    gq = _like("grad_query_out", grad_query_out, query.shape, query)
    gk = _like("grad_key_out", grad_key_out, key.shape, query)
    dq, dk, dwq, dwk = _dense(query), _dense(key), torch.empty_like(wq), torch.empty_like(wk)
    lib = _lib.lib()
    workspace, n = workspace_of(lib.msda_norm_rotary_backward_workspace_size(p), workspace, query.device)
    with on_device(query.device):
        _lib.check(lib.msda_norm_rotary_backward(
            DTYPE_CODE[query.dtype], _lib.ROTARY_INTERLEAVED if interleaved else 0, p, float(eps), ptr(positions),
            ptr(frequencies), ptr(query), ptr(key), ptr(wq), ptr(wk), ptr(gq), ptr(gk), ptr(dq), ptr(dk), ptr(dwq),
            ptr(dwk), ptr(workspace), n, stream(query.device)))
    return dq, dk, dwq, dwk


class _RotaryFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, positions, frequencies, sections, interleaved):
        ctx.save_for_backward(positions, frequencies)
        ctx.how = (sections, interleaved)
        ctx.dtype = x.dtype
        return rotary_forward(x, positions, frequencies, sections, interleaved=interleaved)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        positions, frequencies = ctx.saved_tensors
        sections, interleaved = ctx.how
        return rotary_backward(grad.to(ctx.dtype), positions, frequencies, sections, interleaved=interleaved), None, None, None, None


class _NormRotaryFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, query, key, wq, wk, positions, frequencies, sections, eps, interleaved):
        ctx.save_for_backward(query, key, wq, wk, positions, frequencies)
        ctx.how = (sections, eps, interleaved)
        return norm_rotary_forward(query, key, wq, wk, positions, frequencies, sections, eps=eps,
                                   interleaved=interleaved)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, gq, gk):
        query, key, wq, wk, positions, frequencies = ctx.saved_tensors
        sections, eps, interleaved = ctx.how
        got = norm_rotary_backward(query, key, wq, wk, positions, frequencies, sections, gq.to(query.dtype),
                                   gk.to(query.dtype), eps=eps, interleaved=interleaved)
        return (*got, None, None, None, None, None)


def _no_gradient(positions, frequencies):
    if not torch.is_grad_enabled():
        return
    for name, t in (("positions", positions), ("frequencies", frequencies)):
        if t.requires_grad:
            raise ValueError(f"{name} gets no gradient from this operator: detach it")


def rotary(x: torch.Tensor, positions: torch.Tensor, frequencies: torch.Tensor, sections: Sequence[int],
           interleaved: bool = False) -> torch.Tensor:
    """Differentiable ``rotary_forward``; ``positions`` and ``frequencies`` get no gradient."""
    _no_gradient(positions, frequencies)
    return _RotaryFunction.apply(x, positions, frequencies, tuple(sections), bool(interleaved))


def norm_rotary(query: torch.Tensor, key: torch.Tensor, query_weight: torch.Tensor, key_weight: torch.Tensor,
                positions: torch.Tensor, frequencies: torch.Tensor, sections: Sequence[int], eps: float = 1e-6,
                interleaved: bool = False) -> Tuple[torch.Tensor, torch.Tensor]:
    """Differentiable ``norm_rotary_forward`` (gradients of queries, keys and both weights)."""
    _no_gradient(positions, frequencies)
    return _NormRotaryFunction.apply(query, key, query_weight, key_weight, positions, frequencies, tuple(sections),
                                     float(eps), bool(interleaved))
