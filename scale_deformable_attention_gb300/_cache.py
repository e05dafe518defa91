"""The paged cache of keys and values: writing tokens into it (16 or 32 bits, or quantised to 8), reading them back,
attention of new tokens over it (C ABI ``msda_cache_write`` / ``_read`` / ``_attention``)."""
from __future__ import annotations

import math
from typing import NamedTuple, Optional, Tuple

import torch
from torch.autograd import forward_ad

from . import _lib
from ._binding import DTYPE_CODE, stream, workspace_of

CODE_FORMAT = {torch.float8_e4m3fn: _lib.CACHE_E4M3, torch.int8: _lib.CACHE_INT8}
_NONE3 = (0, 0, 0)


class PagedCache(NamedTuple):
    """``key``, ``value`` [pages, page, N, D] (channels contiguous): float32, float16 or bfloat16, or codes in
    torch.float8_e4m3fn or torch.int8 with ``key_scale``, ``value_scale`` [pages, page, N] uint8: a row is
    code * 2^(byte - 127)."""
    key: torch.Tensor
    value: torch.Tensor
    key_scale: Optional[torch.Tensor] = None
    value_scale: Optional[torch.Tensor] = None


def cache_create(pages: int, page: int, heads: int, channels: int, dtype: torch.dtype = torch.bfloat16,
                 device="cuda") -> PagedCache:
    """A cache of zeros: ``pages`` pages of ``page`` tokens (a power of two, 16 or more), ``channels`` a multiple of 16 up
    to 128; ``dtype`` torch.float8_e4m3fn or torch.int8 for a quantised one.  In memory a page lies head by head, so that
    one head's rows, which an attention block reads, are next to each other."""
    if dtype not in DTYPE_CODE and dtype not in CODE_FORMAT:
        raise TypeError(f"unsupported cache dtype {dtype}; use float32, float16, bfloat16, float8_e4m3fn or int8")
    if pages < 0 or heads < 1 or channels < 16 or channels > 128 or channels % 16 or page < 16 or page & (page - 1):
        raise ValueError(f"pages={pages} of page={page} tokens (a power of two, 16 or more), heads={heads}, "
                         f"channels={channels} (16, 32, ... 128)")
    shape = (pages, heads, page, channels)
    made = [torch.zeros(shape, dtype=dtype, device=device).transpose(1, 2) for _ in range(2)]
    if dtype in CODE_FORMAT:
        made += [torch.zeros(shape[:3], dtype=torch.uint8, device=device).transpose(1, 2) for _ in range(2)]
    return PagedCache(*made)


def _pages(cache: PagedCache):
    """(format, device, [pages, page, N, D], strides, addresses) of a cache, checked."""
    key, value, ks, vs = cache
    sh, dev, dt = key.shape, key.device, key.dtype
    if len(sh) != 4:
        raise ValueError(f"cache.key must be [pages, page, heads, D], got {tuple(sh)}")
    if dev.type != "cuda":
        raise ValueError("the operator runs on CUDA tensors only (there is no CPU implementation)")
    if value.shape != sh or value.dtype is not dt or value.device != dev:
        raise ValueError(f"cache.value must be a {tuple(sh)} {dt} tensor on {dev}")
    k0, k1, k2, k3 = key.stride()
    v0, v1, v2, v3 = value.stride()
    if k3 != 1 or v3 != 1:
        raise ValueError("cache.key and cache.value need contiguous channels")
    if dt in CODE_FORMAT:
        for name, t in (("key_scale", ks), ("value_scale", vs)):
            if t is None or t.shape != sh[:3] or t.dtype is not torch.uint8 or t.device != dev:
                raise ValueError(f"cache.{name} must be a {tuple(sh[:3])} uint8 tensor on {dev}")
        return (CODE_FORMAT[dt], dev, sh, (k0, k1, k2, v0, v1, v2, *ks.stride(), *vs.stride()),
                (key.data_ptr(), value.data_ptr(), ks.data_ptr(), vs.data_ptr()))
    if dt not in DTYPE_CODE:
        raise TypeError(f"unsupported cache dtype {dt}; use float32, float16, bfloat16, float8_e4m3fn or int8")
    if ks is not None or vs is not None:
        raise ValueError(f"a {dt} cache has no scales")
    return _lib.CACHE_SAME, dev, sh, (k0, k1, k2, v0, v1, v2, 0, 0, 0, 0, 0, 0), (key.data_ptr(), value.data_ptr(), None, None)


def _call(f, dev: torch.device, *args):
    """``f(*args, stream)`` with ``dev`` as the current device."""
    if torch.cuda.current_device() == dev.index:
        status = f(*args, stream(dev))
    else:
        with torch.cuda.device(dev):
            status = f(*args, stream(dev))
    if status:
        _lib.check(status)


def _address(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _index(name: str, t: torch.Tensor, B: int, dim: int, dev: torch.device) -> torch.Tensor:
    """An int32 tensor [B] or [B, any] (``dim``) on ``dev`` with contiguous rows."""
    sh = t.shape
    if len(sh) != dim or sh[0] != B:
        raise ValueError(f"{name} must be [{B}{', any' if dim == 2 else ''}], got {tuple(sh)}")
    if t.dtype is not torch.int32:
        raise TypeError(f"{name} must be int32, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, the cache on {dev}")
    return t if sh[-1] <= 1 or t.stride(-1) == 1 else t.contiguous()


def _rows(name: str, x: torch.Tensor, shape, dtype: torch.dtype, dev: torch.device) -> torch.Tensor:
    """``x`` as the kernels read it: rows that begin at multiples of 16 bytes (a copy where they do not)."""
    if x.shape == shape and x.dtype is dtype and x.device == dev and x.is_contiguous() and not x.data_ptr() & 15:
        return x
    if x.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(x.shape)}")
    if x.dtype != dtype:
        raise TypeError(f"{name} is {x.dtype}, expected {dtype}")
    if x.device != dev:
        raise ValueError(f"{name} is on {x.device}, the cache on {dev}")
    if x.data_ptr() % 16 == 0:
        n, st = 16 // x.element_size(), x.stride()
        if st[3] == 1 and all(st[i] % n == 0 or shape[i] <= 1 for i in range(3)):
            return x
    x = x.contiguous()
    return x if x.data_ptr() % 16 == 0 else x.clone()


def _float_dtype(dtype: torch.dtype, fmt: int, cache: PagedCache) -> int:
    if dtype not in DTYPE_CODE:
        raise TypeError(f"unsupported dtype {dtype}; use float32, float16 or bfloat16")
    if fmt == _lib.CACHE_SAME and dtype != cache.key.dtype:
        raise TypeError(f"the tensors are {dtype}, the cache {cache.key.dtype}")
    return DTYPE_CODE[dtype]


def _no_gradient(*tensors):
    reverse, forward = torch.is_grad_enabled(), forward_ad._current_level >= 0
    if not (reverse or forward):
        return
    for t in tensors:
        if t is not None and (reverse and t.requires_grad or forward and forward_ad.unpack_dual(t).tangent is not None):
            raise ValueError("the cache's operators have no gradient: call them under torch.no_grad() or detach the tensors")


def cache_write(cache: PagedCache, key: torch.Tensor, value: torch.Tensor, table: torch.Tensor, start: torch.Tensor, *,
                counts: Optional[torch.Tensor] = None, select: Optional[torch.Tensor] = None) -> PagedCache:
    """Writes tokens into the cache and returns it (C ABI ``msda_cache_write``).

    ``key``, ``value`` [B, T, N, D]; ``table`` [B, width] int32, the page numbers of each sequence; ``start`` [B] int32:
    token r of sequence b becomes its token start[b] + r.  ``counts`` [B] int32: how many tokens of each (all if None).
    ``select`` [B, R] int32: row r is token select[b, r] of ``key`` and ``value``, as for the accepted ones of a drafted tree.
    A quantised cache's rows get the least power of two as scale that brings them into the codes' range.  A place that two
    rows of one call go to holds parts of either in any mixture.
    """
    fmt, dev, sh, strides, places = _pages(cache)
    _no_gradient(cache.key, cache.value, key, value)
    if key.dim() != 4:
        raise ValueError(f"key must be [B, T, heads, D], got {tuple(key.shape)}")
    B, T, N, D = key.shape
    if (N, D) != sh[2:]:
        raise ValueError(f"key has {N} heads of {D} channels, the cache {sh[2]} of {sh[3]}")
    dt = _float_dtype(key.dtype, fmt, cache)
    key, value = _rows("key", key, key.shape, key.dtype, dev), _rows("value", value, key.shape, key.dtype, dev)
    table, start = _index("table", table, B, 2, dev), _index("start", start, B, 1, dev)
    R = T
    if select is not None:
        select = _index("select", select, B, 2, dev)
        R = select.shape[1]
    if counts is not None:
        counts = _index("counts", counts, B, 1, dev)
    width = table.shape[1]
    p = _lib.cache_problem(B, R, N, N, D, T, sh[0], sh[1], width, width * sh[1], *strides, table.stride(0), *_NONE3,
                          *key.stride()[:3], *value.stride()[:3], 0, 0, 0 if select is None else select.stride(0))
    _call(_lib.lib().msda_cache_write, dev, dt, fmt, p, key.data_ptr(), value.data_ptr(), table.data_ptr(), start.data_ptr(),
          _address(counts), _address(select), *places)
    return cache


def cache_read(cache: PagedCache, table: torch.Tensor, lengths: torch.Tensor, rows: int, *,
               dtype: Optional[torch.dtype] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(key, value) [B, rows, N, D]: the first ``rows`` tokens of each sequence, zeros from ``lengths`` [B] (int32) on (C ABI
    ``msda_cache_read``).  ``dtype``: that of the result for a quantised cache (bfloat16 if None)."""
    fmt, dev, sh, strides, places = _pages(cache)
    _no_gradient(cache.key, cache.value)
    if dtype is None:
        dtype = cache.key.dtype if fmt == _lib.CACHE_SAME else torch.bfloat16
    dt = _float_dtype(dtype, fmt, cache)
    if table.dim() != 2:
        raise ValueError(f"table must be [B, width], got {tuple(table.shape)}")
    B, width = table.shape
    table, lengths = _index("table", table, B, 2, dev), _index("lengths", lengths, B, 1, dev)
    key = torch.empty((B, rows, *sh[2:]), dtype=dtype, device=dev)
    value = torch.empty_like(key)
    p = _lib.cache_problem(B, rows, sh[2], sh[2], sh[3], rows, sh[0], sh[1], width, width * sh[1], *strides,
                          table.stride(0), *_NONE3, *_NONE3, *_NONE3, 0, 0, 0)
    _call(_lib.lib().msda_cache_read, dev, dt, fmt, p, *places, table.data_ptr(), lengths.data_ptr(), key.data_ptr(),
          value.data_ptr())
    return key, value


def cache_attention(query: torch.Tensor, cache: PagedCache, table: torch.Tensor, lengths: torch.Tensor,
                    key: Optional[torch.Tensor] = None, value: Optional[torch.Tensor] = None, *,
                    mask: Optional[torch.Tensor] = None, counts: Optional[torch.Tensor] = None,
                    scale: Optional[float] = None, longest: Optional[int] = None,
                    workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(out [B, T, M*D], lse [B, M, T] float32): new tokens over the cache (C ABI ``msda_cache_attention``).

    ``query`` [B, T, M, D] sees the first ``lengths`` [B] (int32) tokens of its sequence in the cache and, where ``key`` and
    ``value`` [B, T, N, D] are given, the new tokens themselves, which need not be in the cache yet: in order (query t sees
    tokens up to t), or by ``mask`` bool [B or 1, T, T] (or [T, T]), True: query t sees token j, as for a tree of drafted
    tokens.  ``counts`` [B] int32: how many of the T tokens a sequence has; what is behind them is padding and gives zeros
    and lse = -inf.  ``scale``: 1 / sqrt(D) if None.  ``longest``: a bound on the lengths that plans the launch (the table's
    width if None).
    """
    fmt, dev, sh, strides, places = _pages(cache)
    _no_gradient(cache.key, cache.value, query, key, value)
    if query.dim() != 4:
        raise ValueError(f"query must be [B, T, heads, D], got {tuple(query.shape)}")
    B, T, M, D = query.shape
    N = sh[2]
    if D != sh[3] or N == 0 or M % N:
        raise ValueError(f"query has {M} heads of {D} channels, the cache {N} (which must divide them) of {sh[3]}")
    dt = _float_dtype(query.dtype, fmt, cache)
    query = _rows("query", query, query.shape, query.dtype, dev)
    table, lengths = _index("table", table, B, 2, dev), _index("lengths", lengths, B, 1, dev)
    width = table.shape[1]
    if longest is None:
        longest = width * sh[1]
    ks = vs = _NONE3
    ms0 = ms1 = 0
    if (key is None) != (value is None):
        raise TypeError("key and value are given together or not at all")
    if key is not None:
        key, value = _rows("key", key, (B, T, N, D), query.dtype, dev), _rows("value", value, (B, T, N, D), query.dtype, dev)
        ks, vs = key.stride()[:3], value.stride()[:3]
    if mask is not None:
        if key is None:
            raise ValueError("mask is of new tokens: it needs key and value")
        if mask.dtype != torch.bool:
            raise TypeError(f"mask must be a bool tensor (True: takes part), got {mask.dtype}")
        if mask.device != dev:
            raise ValueError(f"mask is on {mask.device}, the cache on {dev}")
        if mask.dim() == 2:
            mask = mask[None]
        if tuple(mask.shape) not in ((B, T, T), (1, T, T)):
            raise ValueError(f"mask must be [{B} or 1, T={T}, T={T}], got {tuple(mask.shape)}")
        if T > 1 and mask.stride(2) != 1:
            mask = mask.contiguous()
        ms0, ms1 = 0 if mask.shape[0] == 1 else mask.stride(0), mask.stride(1)
    if counts is not None:
        counts = _index("counts", counts, B, 1, dev)
    p = _lib.cache_problem(B, T, M, N, D, 0 if key is None else T, sh[0], sh[1], width, longest, *strides, table.stride(0),
                          *query.stride()[:3], *ks, *vs, ms0, ms1, 0)
    out = torch.empty((B, T, M * D), dtype=query.dtype, device=dev)
    lse = torch.empty((B, M, T), dtype=torch.float32, device=dev)
    lib = _lib.lib()
    need = lib.msda_cache_attention_workspace_size(dt, fmt, p)
    workspace, n = workspace_of(need, workspace, dev) if need or workspace is not None else (None, 0)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    _call(lib.msda_cache_attention, dev, dt, fmt, p, float(scale), query.data_ptr(), *places, table.data_ptr(),
          lengths.data_ptr(), _address(key), _address(value), _address(mask), _address(counts), out.data_ptr(),
          lse.data_ptr(), _address(workspace), n)
    return out, lse
