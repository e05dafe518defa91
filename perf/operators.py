"""What the dense-attention operators are measured on: rotary positions with
several axes, the norm of queries and keys with that rotation in the same pass,
and softmax attention with its backward pass.

``own`` false computes each operator in plain torch operations in 32 bits
(angles in 64), rounded once to the tensors' type; ``own`` true makes the
framework's calls.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


def _rotary(name, **kw):
    c = dict(op="rotary", dtype="bf16", B=1, S=1, M=8, N=0, D=32, pairs=16, axes=2, interleaved=False,
             positions="pixels", train=False)
    c.update(kw)
    return dict(c, name=name) if name else c


def _attention(name, **kw):
    c = dict(op="attention", dtype="bf16", B=1, Q=1, S=1, M=8, N=8, D=32, mask="none", train=False)
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # 300 object queries of four images get the positions of their reference points (x, y): a latency-bound call
        _rotary("rotary_queries_f32", dtype="f32", B=4, S=300, positions="pixels"),
        # tokens of a clip, eight frames of a 50 x 84 level: axes time, height, width, pairs next to each other, with the gradient
        _rotary("rotary_video_train_bf16", B=4, S=33600, D=64, pairs=32, axes=3, interleaved=True, positions="grid",
                train=True),
        # the queries and keys of a decoder's self-attention
        _rotary("norm_rotary_queries_bf16", op="norm_rotary", B=4, S=300, N=8),
        # every pixel of an 800 x 1333 pyramid as a token, training
        _rotary("norm_rotary_pyramid_train_f16", op="norm_rotary", dtype="f16", B=2, S=22223, N=8, train=True),
        # wide heads with shared keys on a long clip far into a stream (positions of 10^6), training; the largest
        _rotary("norm_rotary_grouped_train_bf16", op="norm_rotary", B=8, S=16641, M=16, N=4, D=128, pairs=56, axes=3,
                positions="far", train=True),
        # self-attention among 300 object queries: a latency-bound call
        _attention("attention_queries_bf16", B=4, Q=300, S=300),
        # one new query over a whole padded pyramid, heads shared in fours
        _attention("attention_single_query_bf16", B=8, Q=1, S=22223, N=2, D=64, mask="keys"),
        # dense encoder attention over a padded pyramid, the forward of an evaluation
        _attention("attention_pyramid_f16", dtype="f16", Q=22223, S=22223, mask="keys"),
        # denoising groups beside the matching queries (a mask of query and key, shared by batch and heads), in binary32 with 48 channels
        _attention("attention_denoising_train_f32", dtype="f32", B=8, Q=900, S=900, D=48, mask="pairs", train=True),
        # the same in 16 bits with more queries
        _attention("attention_denoising_train_bf16", B=4, Q=1100, S=1100, mask="pairs", train=True),
        # frames in order: causal attention on an odd length, wide heads shared in fours
        _attention("attention_causal_train_bf16", B=2, Q=8191, S=8191, M=16, N=4, D=128, mask="causal", train=True),
        # dense encoder attention over a pyramid, training; the largest
        _attention("attention_pyramid_train_f16", dtype="f16", Q=22223, S=22223, D=64, train=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    if rng.random() < 0.4:
        D = rng.choice((16, 32, 48, 64, 96, 128))
        M = rng.choice((1, 4, 8, 16))
        B = _log_int(rng, 1, 8)
        op = rng.choice(("rotary", "norm_rotary"))
        pairs = rng.choice((D // 2, D // 2, 3 * D // 8))
        train = rng.random() < 0.6
        S = _log_int(rng, 1, max(1, min(50000, 340_000_000 // (B * M * D * 3))))
        return _rotary(None, op=op, dtype=dtype, B=B, S=S, M=M, N=0 if op == "rotary" else rng.choice((1, M)), D=D,
                       pairs=pairs, axes=rng.choice((1, 2, 3)), interleaved=rng.random() < 0.5,
                       positions=rng.choice(("pixels", "grid", "far")), train=train)
    D = rng.choice((8, 16, 32, 48, 64, 96, 128))
    M = rng.choice((1, 2, 4, 8, 16))
    N = rng.choice([n for n in (1, 2, 4, 8, 16) if M % n == 0])
    B = _log_int(rng, 1, 8)
    train = rng.random() < 0.5
    mask = rng.choice(("none", "keys", "pairs", "causal"))
    top = 4.0e9 * min(1.0, 64 / D) * (1.0 if dtype != "f32" else 0.2)
    S = _log_int(rng, 1, 22223)
    Q = rng.choice((1, S, S, _log_int(rng, 1, 22223)))
    while float(B) * M * Q * S > top:
        B, Q, S = max(1, B // 2), max(1, Q * 3 // 4), max(1, S * 3 // 4)
    return _attention(None, dtype=dtype, B=B, Q=Q, S=S, M=M, N=N, D=D, mask=mask, train=train)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _sections(pairs, axes):
    """The pairs split over the axes as evenly as they go, the first axes taking what is left over."""
    return tuple(pairs // axes + (1 if a < pairs % axes else 0) for a in range(axes))


def _positions(case, g):
    """Positions [B, S, axes]: points of images in pixels (float32), cells of a grid, or cells far into a stream (int64)."""
    B, S, A = case["B"], case["S"], case["axes"]
    if case["positions"] == "pixels":
        return torch.rand((B, S, A), generator=g, device="cuda") * 1333.0
    n = torch.arange(S, device="cuda")
    wide = max(1, math.isqrt(S) // 2)
    parts = torch.stack((n // (wide * wide), n // wide % wide, n % wide), -1)[:, 3 - A:]
    start = 0 if case["positions"] == "grid" else 1_000_000
    shift = torch.randint(0, 1000, (B, 1, A), generator=g, device="cuda")
    return (parts[None] + shift + start).contiguous()


def _frequencies(case):
    """One frequency a pair, 10000^(-j / pairs of its axis), for each axis."""
    f = [10000.0 ** (-j / n) for n in _sections(case["pairs"], case["axes"]) for j in range(n)]
    return torch.tensor(f, dtype=torch.float32, device="cuda")


def _groups_mask(n):
    """Denoising groups in front, matching queries behind: a group sees itself and the matching queries, these see one another only."""
    matching = max(1, n * 2 // 3)
    size = max(1, (n - matching + 4) // 5)
    i = torch.arange(n, device="cuda")
    group = torch.where(i < n - matching, i // size, -1)
    return (group[None, :] == -1) | (group[:, None] == group[None, :])


def _pair_mask(Q, S, g):
    if Q == S:
        return _groups_mask(Q)
    return torch.rand((Q, S), generator=g, device="cuda") < 0.8


def prepare(case, seed):
    g = _generator(seed)
    dt = DTYPES[case["dtype"]]
    B, S, M, N, D = (case[k] for k in "BSMND")
    st = {"case": case}
    if case["op"] == "attention":
        Q = case["Q"]
        st["query"] = _normal(g, (B, Q, M, D), dt)
        st["key"] = _normal(g, (B, S, N, D), dt)
        st["value"] = _normal(g, (B, S, N, D), dt)
        st["mask"] = _pair_mask(Q, S, g) if case["mask"] == "pairs" else None
        st["key_mask"] = None
        if case["mask"] == "keys":  # the padding of each image: rows behind its last one
            left = torch.randint((S + 1) // 2, S + 1, (B, 1), generator=g, device="cuda")
            st["key_mask"] = torch.arange(S, device="cuda")[None, :] < left
        if case["train"]:
            st["grad_out"] = _normal(g, (B, Q, M * D), dt)
        return st
    st["sections"] = _sections(case["pairs"], case["axes"])
    st["frequencies"] = _frequencies(case)
    st["positions"] = _positions(case, g)
    st["query"] = _normal(g, (B, S, M, D), dt)
    if case["op"] == "norm_rotary":
        st["key"] = _normal(g, (B, S, N, D), dt)
        st["query_weight"] = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(dt)
        st["key_weight"] = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(dt)
    if case["train"]:
        st["grad_query"] = _normal(g, (B, S, M, D), dt)
        if case["op"] == "norm_rotary":
            st["grad_key"] = _normal(g, (B, S, N, D), dt)
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _cos_sin(st):
    """cos and sin [B, S, 1, pairs] of position times frequency, the angle in 64 bits."""
    axes = [a for a, n in enumerate(st["sections"]) for _ in range(n)]
    angle = st["positions"].double()[..., axes] * st["frequencies"].double()
    return torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]


def _rotate(z, cos, sin, pairs, interleaved):
    """z (float32) with its first 2 * pairs channels rotated."""
    if interleaved:
        u, v = z[..., 0:2 * pairs:2], z[..., 1:2 * pairs:2]
        turned = torch.stack((u * cos - v * sin, v * cos + u * sin), -1).flatten(-2)
    else:
        u, v = z[..., :pairs], z[..., pairs:2 * pairs]
        turned = torch.cat((u * cos - v * sin, v * cos + u * sin), -1)
    return torch.cat((turned, z[..., 2 * pairs:]), -1)


def _norm_rotate(x, w, cos, sin, case):
    x32 = x.float()
    r = torch.rsqrt((x32 * x32).mean(-1, keepdim=True) + EPS)
    return _rotate(x32 * r * w.float(), cos, sin, case["pairs"], case["interleaved"]).to(x.dtype)


def _norm_rotate_backward(x, w, dy, cos, sin, case):
    x32 = x.float()
    r = torch.rsqrt((x32 * x32).mean(-1, keepdim=True) + EPS)
    dz = _rotate(dy.float(), cos, -sin, case["pairs"], case["interleaved"])
    dn = dz * w.float()
    n = x32 * r
    dx = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    return dx.to(x.dtype), (dz * n).sum((0, 1, 2)).to(w.dtype)


def _plain_rotary(st):
    case = st["case"]
    cos, sin = _cos_sin(st)
    if case["op"] == "rotary":
        x = st["query"]
        got = {"out": _rotate(x.float(), cos, sin, case["pairs"], case["interleaved"]).to(x.dtype)}
        if case["train"]:
            got["grad"] = _rotate(st["grad_query"].float(), cos, -sin, case["pairs"], case["interleaved"]).to(x.dtype)
        return got
    got = {"query": _norm_rotate(st["query"], st["query_weight"], cos, sin, case),
           "key": _norm_rotate(st["key"], st["key_weight"], cos, sin, case)}
    if case["train"]:
        got["grad_query"], got["grad_query_weight"] = _norm_rotate_backward(
            st["query"], st["query_weight"], st["grad_query"], cos, sin, case)
        got["grad_key"], got["grad_key_weight"] = _norm_rotate_backward(
            st["key"], st["key_weight"], st["grad_key"], cos, sin, case)
    return got


def _allowed(st):
    """Which (query, key) pairs take part, or None for all of them: [B or 1, 1, 1, Q or 1, S]."""
    case = st["case"]
    if case["mask"] == "pairs":
        return st["mask"][None, None, None]
    if case["mask"] == "keys":
        return st["key_mask"][:, None, None, None, :]
    if case["mask"] == "causal":  # the last query sees every key
        i = torch.arange(case["Q"], device="cuda")[:, None] + (case["S"] - case["Q"])
        return (torch.arange(case["S"], device="cuda")[None, :] <= i)[None, None, None]
    return None


def _plain_attention(st):
    case = st["case"]
    B, Q, S, M, N, D = (case[k] for k in ("B", "Q", "S", "M", "N", "D"))
    dt = DTYPES[case["dtype"]]
    scale = 1.0 / math.sqrt(D)
    q = st["query"].float().view(B, Q, N, M // N, D).permute(0, 2, 3, 1, 4)      # [B, N, G, Q, D]
    k = st["key"].float().permute(0, 2, 1, 3)[:, :, None]                         # [B, N, 1, S, D]
    v = st["value"].float().permute(0, 2, 1, 3)[:, :, None]
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(scale)
    allowed = _allowed(st)
    if allowed is not None:
        s.masked_fill_(~allowed, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total))[..., 0].reshape(B, M, Q)
    p.div_(torch.where(total == 0, torch.ones_like(total), total))
    o = torch.matmul(p, v)
    got = {"out": o.permute(0, 3, 1, 2, 4).reshape(B, Q, M * D).to(dt), "lse": lse}
    if case["train"]:
        do = st["grad_out"].float().view(B, Q, N, M // N, D).permute(0, 2, 3, 1, 4)
        delta = (do * o).sum(-1, keepdim=True)
        got["grad_value"] = torch.matmul(p.transpose(-1, -2), do).sum(2).permute(0, 2, 1, 3).to(dt).contiguous()
        ds = torch.matmul(do, v.transpose(-1, -2)).sub_(delta).mul_(p).mul_(scale)
        got["grad_query"] = torch.matmul(ds, k).permute(0, 3, 1, 2, 4).reshape(B, Q, M, D).to(dt)
        got["grad_key"] = torch.matmul(ds.transpose(-1, -2), q).sum(2).permute(0, 2, 1, 3).to(dt).contiguous()
    return got


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _own_rotary(st):
    import scale_deformable_attention_gb300 as msda

    case = st["case"]
    how = (st["positions"], st["frequencies"], st["sections"])
    if case["op"] == "rotary":
        got = {"out": msda.rotary_forward(st["query"], *how, interleaved=case["interleaved"])}
        if case["train"]:
            got["grad"] = msda.rotary_backward(st["grad_query"], *how, interleaved=case["interleaved"])
        return got
    args = (st["query"], st["key"], st["query_weight"], st["key_weight"], *how)
    got = {}
    got["query"], got["key"] = msda.norm_rotary_forward(*args, eps=EPS, interleaved=case["interleaved"])
    if case["train"]:
        (got["grad_query"], got["grad_key"], got["grad_query_weight"],
         got["grad_key_weight"]) = msda.norm_rotary_backward(
            *args, st["grad_query"], st["grad_key"], eps=EPS, interleaved=case["interleaved"])
    return got


def _own_attention(st):
    import scale_deformable_attention_gb300 as msda

    case = st["case"]
    q, k, v = st["query"], st["key"], st["value"]
    how = {"mask": st["mask"], "key_mask": st["key_mask"], "causal": case["mask"] == "causal"}
    out, lse = msda.attention_forward(q, k, v, **how)
    got = {"out": out, "lse": lse}
    if case["train"]:
        got["grad_query"], got["grad_key"], got["grad_value"] = msda.attention_backward(
            q, k, v, out, lse, st["grad_out"], **how)
    return got


def run(state):
    if state["case"]["op"] == "attention":
        return _own_attention(state) if own else _plain_attention(state)
    return _own_rotary(state) if own else _plain_rotary(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    B, S, M, N, D = (case[k] for k in "BSMND")
    if case["op"] != "attention":
        n = B * S * (M + N) * D
        table = B * S * case["axes"] * (4 if case["positions"] == "pixels" else 8) + case["pairs"] * 4
        tensors = 2 if not case["train"] else 4 if case["op"] == "rotary" else 5
        flops = n * (4 if case["op"] == "rotary" else 8) * (2 if case["train"] else 1)
        return {"bytes": n * es * tensors + table, "flops": flops}
    Q = case["Q"]
    pairs = B * M * Q * S
    if case["mask"] == "causal":  # query i sees i + 1 + S - Q keys
        first = max(0, Q - S)
        pairs = B * M * sum_of_seen(Q - first, S)
    elif case["mask"] == "keys":  # between half of the keys and all of them
        pairs = pairs * 3 // 4
    elif case["mask"] == "pairs":
        pairs = pairs * 4 // 5
    qn, kn = B * Q * M * D * es, B * S * N * D * es
    moved = qn * 2 + kn * 2 + B * M * Q * 4
    moved += Q * S if case["mask"] == "pairs" else B * S if case["mask"] == "keys" else 0
    if case["train"]:  # grad_out read, three gradients written
        moved += qn * 2 + kn * 2
    return {"bytes": moved, "flops": pairs * D * (14 if case["train"] else 4)}


def sum_of_seen(rows, S):
    """Keys seen by the last `rows` queries, of which the last sees all S."""
    return rows * S - rows * (rows - 1) // 2


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _exact_rotation(case, st):
    """The rotation as complex numbers e^(i t), one for each pair."""
    pos = st["positions"].double()
    f = st["frequencies"].double()
    t, j = [], 0
    for a, n in enumerate(st["sections"]):
        t.append(pos[:, :, a, None] * f[j:j + n])
        j += n
    t = torch.cat(t, -1)[:, :, None]
    return torch.polar(torch.ones_like(t), t)


def _exact_turn(z, e, case):
    P = case["pairs"]
    out = z.clone()
    one, two = (slice(0, 2 * P, 2), slice(1, 2 * P, 2)) if case["interleaved"] else (slice(0, P), slice(P, 2 * P))
    c = torch.complex(z[..., one].contiguous(), z[..., two].contiguous()) * e
    out[..., one], out[..., two] = c.real, c.imag
    return out


def _exact_norm(x, w, dy, e, case):
    """Output, and with dy the gradients, one batch item at a time."""
    ys, dxs, dw = [], [], torch.zeros(case["D"], dtype=torch.float64, device="cuda")
    w = w.double()
    for b in range(x.shape[0]):
        xb = x[b:b + 1].double()
        r = ((xb ** 2).sum(-1, keepdim=True) / case["D"] + EPS) ** -0.5
        ys.append(_exact_turn(xb * r * w, e[b:b + 1], case))
        if dy is not None:
            dz = _exact_turn(dy[b:b + 1].double(), e[b:b + 1].conj(), case)
            dw += (dz * xb * r).sum((0, 1, 2))
            dxs.append(dz * w * r - xb * r ** 3 * (dz * w * xb).sum(-1, keepdim=True) / case["D"])
    return torch.cat(ys), torch.cat(dxs) if dxs else None, dw


def _exact_attention(case, st):
    B, Q, S, M, N, D = (case[k] for k in ("B", "Q", "S", "M", "N", "D"))
    train, scale = case["train"], D ** -0.5
    dev = {"dtype": torch.float64, "device": "cuda"}
    out, lse = torch.zeros((B, Q, M, D), **dev), torch.empty((B, M, Q), **dev)
    dq, dk, dv = torch.zeros((B, Q, M, D), **dev), torch.zeros((B, S, N, D), **dev), torch.zeros((B, S, N, D), **dev)
    rows = max(1, min(Q, 200_000_000 // S))
    cols = torch.arange(S, device="cuda")
    for b in range(B):
        for m in range(M):
            n = m // (M // N)
            k, v = st["key"][b, :, n].double(), st["value"][b, :, n].double()
            for i in range(0, Q, rows):
                at = slice(i, min(Q, i + rows))
                q = st["query"][b, at, m].double()
                s = q @ k.T * scale
                if case["mask"] == "pairs":
                    s[~st["mask"][at]] = -math.inf
                elif case["mask"] == "keys":
                    s[:, ~st["key_mask"][b]] = -math.inf
                elif case["mask"] == "causal":
                    last = torch.arange(at.start, at.stop, device="cuda") + S - Q
                    s[cols[None] > last[:, None]] = -math.inf
                z = torch.logsumexp(s, -1, keepdim=True)
                p = torch.exp(s - torch.where(z == -math.inf, 0.0, z))
                out[b, at, m], lse[b, m, at] = p @ v, z[:, 0]
                if train:
                    do = st["grad_out"][b, at].reshape(-1, M, D)[:, m].double()
                    dv[b, :, n] += p.T @ do
                    dp = do @ v.T
                    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * scale
                    dq[b, at, m] = ds @ k
                    dk[b, :, n] += ds.T @ q
    got = {"out": out.view(B, Q, M * D), "lse": lse}
    if train:
        got.update(grad_query=dq, grad_key=dk, grad_value=dv)
    return got


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "attention":
        # about 1 TFLOP/s in binary64
        return _exact_attention(case, st) if work(case)["flops"] < 8e12 else None
    e = _exact_rotation(case, st)
    if case["op"] == "rotary":
        got = {"out": _exact_turn(st["query"].double(), e, case)}
        if case["train"]:
            got["grad"] = _exact_turn(st["grad_query"].double(), e.conj(), case)
        return got
    got = {}
    got["query"], dq, dqw = _exact_norm(st["query"], st["query_weight"], st.get("grad_query"), e, case)
    got["key"], dk, dkw = _exact_norm(st["key"], st["key_weight"], st.get("grad_key"), e, case)
    if case["train"]:
        got.update(grad_query=dq, grad_query_weight=dqw, grad_key=dk, grad_key_weight=dkw)
    return got
