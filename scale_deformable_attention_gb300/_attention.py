"""Dense softmax attention and its gradients (C ABI ``msda_attention_forward`` / ``_backward``)."""
from __future__ import annotations

import math
from typing import Optional, Tuple

import torch

from . import _lib
from ._binding import DTYPE_CODE, on_device, ptr, stream, workspace_of


def _rows(name: str, x: torch.Tensor) -> torch.Tensor:
    """``x`` [B, rows, heads, D] as the kernels read it: channels contiguous,
    every other stride at least a row (a broadcast dimension is copied)."""
    if x.is_contiguous() and x.dim() == 4:
        return x
    if x.dim() != 4:
        raise ValueError(f"{name} must be [B, rows, heads, D], got shape {tuple(x.shape)}")
    st, sh = x.stride(), x.shape
    if (st[3] != 1 and sh[3] > 1) or any(st[i] == 0 and sh[i] > 1 for i in range(3)):
        return x.contiguous()
    return x


def _byte_mask(name: str, m: torch.Tensor, dev: torch.device) -> torch.Tensor:
    if m.dtype != torch.bool:
        raise TypeError(f"{name} must be a bool tensor (True: takes part), got {m.dtype}")
    if m.device != dev:
        raise ValueError(f"{name} is on {m.device}, query on {dev}")
    return m if m.shape[-1] <= 1 or m.stride(-1) == 1 else m.contiguous()


def _problem(query, key, value, mask, key_mask, causal, scale):
    """Checks, and the C ABI's arguments: (query, key, value, mask, key_mask, flags, problem, scale, dims)."""
    query, key, value = _rows("query", query), _rows("key", key), _rows("value", value)
    B, Q, M, D = query.shape
    S, N = key.shape[1], key.shape[2]
    if query.dtype not in DTYPE_CODE:
        raise TypeError(f"unsupported dtype {query.dtype}; use float32, float16 or bfloat16")
    dev = query.device
    if dev.type != "cuda":
        raise ValueError("the operator runs on CUDA tensors only (there is no CPU implementation)")
    for name, t in (("key", key), ("value", value)):
        if t.shape != (B, S, N, D):
            raise ValueError(f"{name} must be [B={B}, S={S}, heads={N}, D={D}], got {tuple(t.shape)}")
        if t.dtype != query.dtype:
            raise TypeError(f"{name} is {t.dtype}, query {query.dtype}; all float tensors share one dtype")
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, query on {dev}")
    if N == 0 or M % N:
        raise ValueError(f"the {N} key heads must divide the {M} query heads")
    flags = _lib.ATTENTION_CAUSAL if causal else 0
    ms, kms = (0, 0, 0), 0
    if mask is not None:
        if mask.dim() > 4 or mask.dim() < 2:
            raise ValueError(f"mask must be [Q, S], or with heads and a batch in front, got {tuple(mask.shape)}")
        mask = _byte_mask("mask", mask, dev)
        while mask.dim() < 4:
            mask = mask[None]
        sh = tuple(mask.shape)
        if sh[0] not in (1, B) or sh[1] not in (1, M) or sh[2] not in (1, Q) or sh[3] != S:
            raise ValueError(f"mask must be [{B} or 1, {M} or 1, {Q} or 1, S={S}], got {sh}")
        ms = tuple(0 if sh[i] == 1 else mask.stride(i) for i in range(3))
        flags |= _lib.ATTENTION_MASK
    if key_mask is not None:
        if tuple(key_mask.shape) not in ((B, S), (1, S)):
            raise ValueError(f"key_mask must be [{B} or 1, S={S}], got {tuple(key_mask.shape)}")
        key_mask = _byte_mask("key_mask", key_mask, dev)
        kms = 0 if key_mask.shape[0] == 1 else key_mask.stride(0)
        flags |= _lib.ATTENTION_KEY_MASK
    qs, ks, vs = query.stride(), key.stride(), value.stride()
    p = _lib.AttentionProblem(B, Q, S, M, N, D, qs[0], qs[1], qs[2], ks[0], ks[1], ks[2], vs[0], vs[1], vs[2], kms, *ms)
    if scale is None:
        scale = 1.0 / math.sqrt(D) if D else 1.0
    return query, key, value, mask, key_mask, flags, p, float(scale), (B, Q, S, M, N, D)


def attention_forward(query: torch.Tensor, key: torch.Tensor, value: torch.Tensor, *,
                      mask: Optional[torch.Tensor] = None, key_mask: Optional[torch.Tensor] = None,
                      causal: bool = False, scale: Optional[float] = None, workspace: Optional[torch.Tensor] = None
                      ) -> Tuple[torch.Tensor, torch.Tensor]:
    """(out [B, Q, M*D], lse [B, M, Q] float32) on the current stream (C ABI ``msda_attention_forward``).

    ``query`` [B, Q, M, D]; ``key``, ``value`` [B, S, N, D] with N dividing M (M / N heads share a key head).
    ``mask`` bool [B or 1, M or 1, Q or 1, S] (or without the leading dimensions) and ``key_mask`` bool
    [B or 1, S]: True takes part.  ``causal``: query i sees keys up to i + S - Q.  ``scale``: 1 / sqrt(D) if None.
    A query that sees no key gives zeros and lse = -inf.
    """
    query, key, value, mask, key_mask, flags, p, scale, (B, Q, S, M, N, D) = _problem(query, key, value, mask,
                                                                                      key_mask, causal, scale)
    dev = query.device
    out = torch.empty((B, Q, M * D), dtype=query.dtype, device=dev)
    lse = torch.empty((B, M, Q), dtype=torch.float32, device=dev)
    lib, dt = _lib.lib(), DTYPE_CODE[query.dtype]
    workspace, n = workspace_of(lib.msda_attention_forward_workspace_size(dt, flags, p), workspace, dev)
    with on_device(dev):
        _lib.check(lib.msda_attention_forward(dt, flags, p, scale, ptr(query), ptr(key), ptr(value), ptr(key_mask),
                                              ptr(mask), ptr(out), ptr(lse), ptr(workspace), n, stream(dev)))
    return out, lse


def attention_backward(query: torch.Tensor, key: torch.Tensor, value: torch.Tensor, out: torch.Tensor,
                       lse: torch.Tensor, grad_out: torch.Tensor, *, mask: Optional[torch.Tensor] = None,
                       key_mask: Optional[torch.Tensor] = None, causal: bool = False, scale: Optional[float] = None,
                       workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(grad_query, grad_key, grad_value) (C ABI ``msda_attention_backward``): the probabilities are recomputed from
    the forward's ``out`` and ``lse``; masks and scale as given to the forward."""
    query, key, value, mask, key_mask, flags, p, scale, (B, Q, S, M, N, D) = _problem(query, key, value, mask,
                                                                                      key_mask, causal, scale)
    dev = query.device
    for name, t in (("out", out), ("grad_out", grad_out)):
        if tuple(t.shape) != (B, Q, M * D) or t.dtype != query.dtype or t.device != dev:
            raise ValueError(f"{name} must be a [B, Q, M*D] {query.dtype} tensor on {dev}")
    if tuple(lse.shape) != (B, M, Q) or lse.dtype != torch.float32 or lse.device != dev:
        raise ValueError(f"lse must be a [B, M, Q] float32 tensor on {dev}")
    out, lse, grad_out = out.contiguous(), lse.contiguous(), grad_out.contiguous()
    gq = torch.empty((B, Q, M, D), dtype=query.dtype, device=dev)
    gk = torch.empty((B, S, N, D), dtype=query.dtype, device=dev)
    gv = torch.empty((B, S, N, D), dtype=query.dtype, device=dev)
    lib, dt = _lib.lib(), DTYPE_CODE[query.dtype]
    workspace, n = workspace_of(lib.msda_attention_backward_workspace_size(dt, flags, p), workspace, dev)
    with on_device(dev):
        _lib.check(lib.msda_attention_backward(dt, flags, p, scale, ptr(query), ptr(key), ptr(value), ptr(key_mask),
                                               ptr(mask), ptr(out), ptr(lse), ptr(grad_out), ptr(gq), ptr(gk), ptr(gv),
                                               ptr(workspace), n, stream(dev)))
    return gq, gk, gv


class _AttentionFunction(torch.autograd.Function):
    """Saves the inputs, the output and each row's lse; the backward recomputes the probabilities."""

    @staticmethod
    def forward(ctx, query, key, value, mask, key_mask, causal, scale):
        out, lse = attention_forward(query, key, value, mask=mask, key_mask=key_mask, causal=causal, scale=scale)
        ctx.save_for_backward(query, key, value, out, lse, mask, key_mask)
        ctx.how = (causal, scale)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_out):
        query, key, value, out, lse, mask, key_mask = ctx.saved_tensors
        causal, scale = ctx.how
        got = attention_backward(query, key, value, out, lse, grad_out.to(query.dtype), mask=mask, key_mask=key_mask,
                                 causal=causal, scale=scale)
        return (*got, None, None, None, None)


def attention(query: torch.Tensor, key: torch.Tensor, value: torch.Tensor, mask: Optional[torch.Tensor] = None,
              key_mask: Optional[torch.Tensor] = None, causal: bool = False, scale: Optional[float] = None
              ) -> torch.Tensor:
    """Differentiable ``attention_forward``: out [B, Q, M*D], the layout of the sampled attention's output."""
    return _AttentionFunction.apply(query, key, value, mask, key_mask, bool(causal), scale)
