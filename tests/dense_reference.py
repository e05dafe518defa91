"""Attention, rotary positions and their gradients in 64 bits with elementary
torch operations, and how far a kernel may be from them.

Tolerances are bounds, worked out value by value from the same inputs: ``u`` is
half a step of the tensors' type (``finfo.eps / 2``), ``f`` half a step of
binary32 with a factor two for sums that a matrix unit may truncate, and each
sum of n terms is off by at most n f times the sum of the terms' sizes.
"""
import math

import torch

F = 2.0 ** -23


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rounded(x, e, dtype):
    """Bound of a value ``x`` computed within ``e`` and rounded once to ``dtype``: half a step relative to the computed
    value, and below the type's normal range half of its smallest step, tiny * eps / 2 (binary16: 2^-25), where the
    steps stop shrinking with the value."""
    i = torch.finfo(dtype)
    return e + i.eps / 2 * (x.abs() + e) + i.tiny * i.eps / 2


def attention(q, k, v, do=None, allowed=None, scale=None):
    """q [B, Q, M, D], k and v [B, S, N, D], do [B, Q, M*D], allowed bool broadcast to [B, M, Q, S] or None.
    Returns {name: (value, bound)} with the bounds for tensors of q's dtype."""
    B, Q, M, D = q.shape
    S, N = k.shape[1], k.shape[2]
    G, dt = M // N, q.dtype
    u = half_step(dt)
    up = u if dt != torch.float32 else 0.0        # the probabilities' rounding before their product
    scale = 1 / math.sqrt(D) if scale is None else scale
    q64 = q.double().transpose(1, 2)
    dead = None
    if allowed is not None:
        allowed = allowed.expand(B, M, Q, S)
        seen = allowed.reshape(B, N, G, Q, S).any(3).any(2)          # keys that some query sees
        dead = ~seen.transpose(1, 2)[..., None]
    k64, v64 = k.double(), v.double()
    if dead is not None:
        k64, v64 = k64.masked_fill(dead, 0), v64.masked_fill(dead, 0)
    k64 = k64.transpose(1, 2).repeat_interleave(G, 1)
    v64 = v64.transpose(1, 2).repeat_interleave(G, 1)
    empty = torch.zeros((B, M, Q, 1), dtype=torch.bool, device=q.device) if S else torch.ones(
        (B, M, Q, 1), dtype=torch.bool, device=q.device)
    if allowed is not None and S:
        empty = ~allowed.any(-1, keepdim=True)
    q64 = q64.masked_fill(empty, 0)
    s = scale * (q64 @ k64.transpose(-1, -2))
    # scores: the product's sum, the scaling, the difference to the row's maximum
    es = (D + 6) * F * scale * (q64.abs() @ k64.abs().transpose(-1, -2)) + 4 * F * (s.abs() + 1)
    if allowed is not None:
        s = s.masked_fill(~allowed, -math.inf)
        es = es.masked_fill(~allowed, 0)
    lse = torch.logsumexp(s, -1, keepdim=True) if S else torch.full_like(empty, -math.inf, dtype=torch.float64)
    p = torch.where(empty, 0.0, torch.exp(s - torch.where(empty, 0.0, lse)))
    o = p @ v64
    top = es.amax(-1, keepdim=True) if S else torch.zeros_like(lse)
    rp = es + top + (S + 64) * F                  # relative error of a probability
    eo = (p * (rp + up)) @ v64.abs() + (S + 8) * F * (p @ v64.abs())
    to = lambda x: x.transpose(1, 2)              # noqa: E731
    got = {"out": (to(o).reshape(B, Q, M * D), to(rounded(o, eo, dt)).reshape(B, Q, M * D)),
           "lse": (lse[..., 0], (top + (S + 64) * F + 4 * F * torch.where(empty, 0.0, lse).abs())[..., 0])}
    if do is None:
        return got
    g = do.double().view(B, Q, M, D).transpose(1, 2).masked_fill(empty, 0)
    dp = g @ v64.transpose(-1, -2)
    edp = (D + 6) * F * (g.abs() @ v64.abs().transpose(-1, -2))
    delta = (g * o).sum(-1, keepdim=True)
    ed = (g.abs() * rounded(o, eo, dt)).sum(-1, keepdim=True) + (D + 6) * F * (g * o).abs().sum(-1, keepdim=True)
    ds = p * (dp - delta)
    rp = rp + 4 * F * torch.where(empty, 0.0, lse).abs()
    eds = p * (1 + rp) * (edp + ed + 2 * F * (dp.abs() + delta.abs())) + ds.abs() * (rp + up)
    if dt == torch.float16:                       # what the type's smallest step leaves of scaled values
        eds = eds + 2.0 ** -36 * (dp.abs() + delta.abs()).amax().clamp(min=1e-30) * (p > 0)
    ep = p * (rp + up) + (2.0 ** -36 if dt == torch.float16 else 0.0) * (p > 0)
    share = lambda x: x.reshape(B, N, G, S, D).sum(2).transpose(1, 2)   # noqa: E731
    rows = Q * G
    done = lambda x, e, n, a: (x, rounded(x, e + (n + 8) * F * a, dt))   # noqa: E731
    got["grad_value"] = done(share(p.transpose(-1, -2) @ g), share(ep.transpose(-1, -2) @ g.abs()), rows,
                             share(p.transpose(-1, -2) @ g.abs()))
    got["grad_query"] = done(to(scale * (ds @ k64)), to(scale * (eds @ k64.abs())), S,
                             to(scale * (ds.abs() @ k64.abs())))
    got["grad_key"] = done(share(scale * (ds.transpose(-1, -2) @ q64)), share(scale * (eds.transpose(-1, -2) @ q64.abs())),
                           rows, share(scale * (ds.abs().transpose(-1, -2) @ q64.abs())))
    return got


def turn(z, positions, frequencies, sections, interleaved, inverse=False):
    """z (64 bits) [B, S, H, D] with its pairs turned."""
    axes = [a for a, n in enumerate(sections) for _ in range(n)]
    t = positions.double()[..., axes] * frequencies.double()
    t = (-t if inverse else t)[:, :, None]
    P = len(axes)
    out = z.clone()
    one, two = (slice(0, 2 * P, 2), slice(1, 2 * P, 2)) if interleaved else (slice(0, P), slice(P, 2 * P))
    u, v = z[..., one], z[..., two]
    out[..., one] = u * torch.cos(t) - v * torch.sin(t)
    out[..., two] = v * torch.cos(t) + u * torch.sin(t)
    return out


def pair_size(z, P, interleaved):
    """|u| + |v| of each channel's pair (the size that an angle's error multiplies); |z| behind the pairs."""
    a = z.abs()
    out = a.clone()
    one, two = (slice(0, 2 * P, 2), slice(1, 2 * P, 2)) if interleaved else (slice(0, P), slice(P, 2 * P))
    out[..., one] = out[..., two] = a[..., one] + a[..., two]
    return out


# an angle (product, reduction in three parts, sincosf at two steps) and the rotation's three roundings
TURN = 16 * 2.0 ** -24


def norm_rotary(x, w, positions, frequencies, sections, interleaved, eps, dy=None):
    """{name: (value, bound)} of the norm with rotation of one tensor."""
    P, D = sum(sections), x.shape[3]
    x64 = x.double()
    z, n, r = x64, None, None
    if w is not None:
        r = (x64.square().mean(-1, keepdim=True) + eps) ** -0.5
        n = x64 * r
        z = n * w.double()
    rel = (D + 16) * 2.0 ** -24 if w is not None else 0.0       # the row's sum, rsqrt, two products
    y = turn(z, positions, frequencies, sections, interleaved)
    e = (TURN + 2 * rel) * pair_size(z, P, interleaved)
    got = {"out": (y, rounded(y, e, x.dtype))}
    if dy is None:
        return got
    dz = turn(dy.double(), positions, frequencies, sections, interleaved, inverse=True)
    edz = TURN * pair_size(dy.double(), P, interleaved)
    if w is None:
        got["grad"] = (dz, rounded(dz, edz, x.dtype))
        return got
    g = dz * w.double()
    dot = (g * n).mean(-1, keepdim=True)
    dx = r * (g - n * dot)
    eg = edz * w.double().abs() + 2 * 2.0 ** -24 * g.abs()
    edot = (eg * n.abs()).mean(-1, keepdim=True) + (D + 8 + 2 * rel / 2.0 ** -24) * 2.0 ** -24 * (g * n).abs().mean(-1, keepdim=True)
    edx = r * (eg + n.abs() * edot) + (3 * rel + 8 * 2.0 ** -24) * r * (g.abs() + (n * dot).abs())
    got["grad"] = (dx, rounded(dx, edx, x.dtype))
    dw = (dz * n).sum((0, 1, 2))
    rows = x.shape[0] * x.shape[1] * x.shape[2]
    edw = (edz * n.abs()).sum((0, 1, 2)) + ((rows + 8) * 2.0 ** -24 + 2 * rel) * (dz * n).abs().sum((0, 1, 2))
    got["grad_weight"] = (dw, rounded(dw, edw, x.dtype))
    return got


def check(got, want, what):
    value, bound = want
    got, value, bound = got.detach().double().reshape(value.shape), value.detach(), bound.detach()
    same = torch.equal(torch.isneginf(got), torch.isneginf(value))
    assert same, f"{what}: -inf in other places"
    fine = ~torch.isneginf(value)
    off = (got - value).abs()[fine]
    over = off > bound.expand(value.shape)[fine] + 1e-30
    worst = float((off / (bound.expand(value.shape)[fine] + 1e-30)).max()) if off.numel() else 0.0
    assert not torch.isnan(off).any(), f"{what}: NaN in {int(torch.isnan(off).sum())} places"
    assert not over.any(), f"{what}: {int(over.sum())} of {over.numel()} values off by more than their bound (worst {worst:.3g} bounds)"
    return worst
