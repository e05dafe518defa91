"""The paged cache in 64 bits with elementary operations, and how far the kernels may be from it.

Attention: per sequence the dense reference over the values that the cache stands for.  Beyond its bounds come what
probabilities lose that are held in f16 (f16 queries, quantised caches): 2^-30 of a row's largest, for each key, times the
largest value (in a quantised cache a probability is held times its key's scale over the largest scale).
"""
import math

import torch

import dense_reference as R

MOST = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
FORMAT = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def power(e):
    """2^e in 64 bits, put together from its bits (a power function may be off in the last place)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def exponent(top, most):
    """Least e >= -100 with top <= most 2^e (top > 0)."""
    m, e = torch.frexp(top / most)                  # exact: top is a binary32 value; the quotient is rounded, so look again
    e = e.to(torch.int32) - 1
    e = torch.where(top > most * power(e), e + 1, e)
    e = torch.where(top > most * power(e), e + 1, e)
    return e.clamp(min=-100)


def quantise(x, fmt):
    """(codes in 64 bits, bytes) of rows x."""
    most = MOST[fmt]
    x = x.double()
    top = x.abs().amax(-1)
    fine = top.isfinite()
    e = exponent(torch.where(fine & (top > 0), top, 1.0), most)
    e = torch.where(top > 0, e, -100)
    y = torch.where(fine[..., None], x / power(e)[..., None], 0.0)
    if fmt == torch.int8:
        codes = torch.round(y)
    else:                                           # three binary places behind the first, down to 2^-9
        _, p = torch.frexp(y)
        step = power((p.to(torch.int32) - 1).clamp(min=-6) - 3)
        codes = torch.round(y / step) * step
    return codes, torch.where(fine, e + 127, 255)


def stands_for(codes, scale):
    """Values in 64 bits of a cache's rows (codes, or the rows themselves where scale is None)."""
    if scale is None:
        return codes.double()
    s = power(scale.to(torch.int32) - 127)
    s = torch.where(scale == 255, math.nan, torch.where(scale == 0, 0.0, s))
    return codes.float().double() * s[..., None]


def tokens(cache, table, b, n):
    """The first n tokens of sequence b: (key, value) in 64 bits [n, N, D]."""
    page = cache.key.shape[1]
    at = torch.arange(n, device=table.device)
    block, place = table[b].long()[at // page], at % page

    def rows(x, s):
        bits = x.view(torch.uint8) if x.element_size() == 1 else x
        return stands_for(bits[block, place].view(x.dtype), None if s is None else s[block, place])
    return rows(cache.key, cache.key_scale), rows(cache.value, cache.value_scale)


def attention(q, cache, table, lengths, key=None, value=None, mask=None, counts=None, scale=None):
    """{name: (value, bound)} of cache_attention."""
    B, T, M, D = q.shape
    dev = q.device
    half = q.dtype == torch.float16 or cache.key_scale is not None
    out, eo = torch.zeros((2, B, T, M * D), dtype=torch.float64, device=dev)
    lse, el = torch.full((B, M, T), -math.inf, dtype=torch.float64, device=dev), torch.zeros((B, M, T), dtype=torch.float64, device=dev)
    for b in range(B):
        n = int(lengths[b])
        c = T if counts is None else int(counts[b])
        if c == 0:
            continue
        k, v = tokens(cache, table, b, n)
        ok = torch.ones((c, n), dtype=torch.bool, device=dev)
        if key is not None:
            k, v = torch.cat((k, key[b, :c].double())), torch.cat((v, value[b, :c].double()))
            mine = torch.ones((c, c), dtype=torch.bool, device=dev).tril()
            if mask is not None:
                m3 = mask if mask.dim() == 3 else mask[None]
                mine = m3[b if m3.shape[0] > 1 else 0, :c, :c]
            ok = torch.cat((ok, mine), 1)
        if k.shape[0] == 0:
            continue
        want = R.attention(q[b:b + 1, :c], k[None], v[None], None, ok[None, None], scale)
        o, e = want["out"]
        if half:
            e = e + 2.0 ** -30 * k.shape[0] * v.abs().amax()
        out[b, :c], eo[b, :c] = o[0], e[0]
        lse[b, :, :c], el[b, :, :c] = want["lse"][0][0], want["lse"][1][0]
    return {"out": (out, eo), "lse": (lse, el)}
