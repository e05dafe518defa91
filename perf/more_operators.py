"""What the operators of the paged cache are measured on: tokens quantised as
they are written into its pages, read back from them, and the attention of new
tokens (one, a tree of drafted ones, a piece of a prompt) over it.

``own`` false computes each operator in plain torch operations in 32 bits,
rounded once to the tensors' type; ``own`` true makes the framework's calls.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
# of a row's largest magnitude m 2^e (1/2 <= m < 1): the exponent of its scale is e - PLACES, one more where m is above MOST
PLACES = {"e4m3": 9, "int8": 7}
MOST = {"e4m3": 448 / 512, "int8": 127 / 128}
LEAST = -100  # the smallest exponent of a scale


def _attention(name, **kw):
    c = dict(op="attention", dtype="bf16", cache="same", B=1, T=1, S=1, M=8, N=8, D=64, page=64, new="chain",
             lengths="half", counts="all")
    c.update(kw)
    return dict(c, name=name) if name else c


def _write(name, **kw):
    c = dict(op="write", dtype="bf16", cache="same", B=1, T=1, R=1, S=0, N=8, D=64, page=64, select=False,
             counts="all")
    c.update(kw)
    return dict(c, name=name) if name else c


def _read(name, **kw):
    c = dict(op="read", dtype="bf16", cache="e4m3", B=1, S=1, N=8, D=64, page=64, lengths="half")
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one new token of four short sequences: a latency-bound call
        _attention("token_short_bf16", B=4, S=300, D=32, page=16),
        # one new token over the tokens of whole pyramids, in 8 bits, heads shared in fours
        _attention("token_pyramid_e4m3", cache="e4m3", B=8, S=22223, N=2),
        # one new token far into two streams of clips (four of 33600 tokens), wide heads shared in fours
        _attention("token_stream_f16", dtype="f16", B=2, S=134400, M=16, N=4, D=128, page=256),
        # a small tree of drafted tokens in binary32, 48 channels
        _attention("tree_small_f32", dtype="f32", B=8, T=25, S=900, D=48, page=32, new="tree", counts="ragged"),
        # a tree of 16 drafted tokens, wide heads shared in fours, in 8 bits
        _attention("tree_grouped_int8", cache="int8", B=16, T=16, S=16641, M=16, N=4, D=128, new="tree"),
        # a wide tree over an unquantised cache; the largest
        _attention("tree_wide_bf16", B=8, T=64, S=22223, M=16, N=4, D=128, page=128, new="tree", counts="ragged"),
        # a piece of a prompt, an odd length in order, behind what the cache holds
        _attention("piece_e4m3_f16", dtype="f16", cache="e4m3", B=2, T=1100, S=8191, page=32),
        # the new token of 32 sequences goes into the cache: a latency-bound call
        _write("write_token_bf16", B=32, S=900, page=16),
        # prompts quantised into the cache and read back
        _write("write_prompt_e4m3", cache="e4m3", B=8, T=16641, R=16641, N=4, D=128, counts="ragged"),
        # the accepted tokens of drafted trees, behind what the cache holds, and the sequences read back
        _write("write_accepted_int8", dtype="f16", cache="int8", B=16, T=64, R=9, S=300, page=32, select=True,
               counts="ragged"),
        # sequences of odd lengths read back in binary32
        _read("read_ragged_int8_f32", dtype="f32", cache="int8", B=4, S=8191, D=48, page=16, lengths="any"),
        # whole pyramids read back
        _read("read_pyramid_e4m3", B=8, S=22223),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6.8e12, w["flops"] / 4e14)


def draw(rng):
    op = rng.choice(("attention", "attention", "attention", "write", "read"))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    M = rng.choice((1, 2, 4, 8, 16))
    how = dict(dtype=dtype, cache=rng.choice(("same", "e4m3", "int8")), B=_log_int(rng, 1, 32),
               D=rng.choice((16, 32, 48, 64, 80, 96, 128)), page=rng.choice((16, 32, 64, 128, 256)),
               N=rng.choice([n for n in (1, 2, 4, 8, 16) if M % n == 0]))
    most = 240e-6
    if op == "read":
        c = _read(None, **how, S=_log_int(rng, 1, 33600), lengths=rng.choice(("full", "half", "any")))
    elif op == "write":
        T = _log_int(rng, 1, 22223)
        select = T <= 300 and rng.random() < 0.5
        c = _write(None, **how, T=T, R=max(1, T // 4) if select else T, S=rng.choice((0, _log_int(rng, 1, 900))),
                   select=select, counts=rng.choice(("all", "ragged")))
    else:
        new = rng.choice(("none", "chain", "chain", "tree"))
        T = rng.choice((1, _log_int(rng, 1, 64), _log_int(rng, 1, 1100) if new == "chain" else 8))
        c = _attention(None, **how, M=M, T=T, S=_log_int(rng, 1, 33600), new=new,
                       lengths=rng.choice(("full", "half", "any")), counts=rng.choice(("all", "ragged")))
        most = 240e-6 if dtype != "f32" else 60e-6
    while _cost(c) > most:
        c["B"] = max(1, c["B"] // 2)
        if "S" in c:
            c["S"] = c["S"] * 3 // 4
        if c["op"] == "write":
            c["T"] = max(1, c["T"] * 3 // 4)
            c["R"] = min(c["R"], c["T"])
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _lengths(case):
    """Tokens that each sequence has in the cache: of its sizes alone, so that the work is known."""
    B, S = case["B"], case["S"]
    if case.get("lengths", "full") == "full":
        return [S] * B
    part = [((b * 7 + 3) % 16) / 15 for b in range(B)]      # 0.2 first; 1 and 0 among the first nine
    least = S // 2 if case["lengths"] == "half" else 0
    return [S if b == 0 else least + int((S - least) * part[b]) for b in range(B)]


def _counts(case):
    """New tokens of each sequence, the first having all."""
    B, n = case["B"], case["R"] if case["op"] == "write" else case["T"]
    if case["counts"] == "all":
        return [n] * B
    return [n if b == 0 else 1 + (n - 1) * ((b * 5 + 2) % 8) // 8 for b in range(B)]


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _pool(case, rows, g, fill):
    """Pages [pages, page, N, D] (in memory head by head) that hold `rows` tokens of each sequence, at places in any
    order, with scales if quantised; the table [B, W] of the pages of each sequence."""
    B, N, D, page = (case[k] for k in ("B", "N", "D", "page"))
    W = max(1, -(-rows // page))
    pages = B * W + 3
    table = torch.randperm(pages, generator=g, device="cuda")[:B * W].view(B, W).int()
    shape = (pages, N, page, D)
    pool = {}
    for name in ("key", "value"):
        x = torch.randn(shape, generator=g, device="cuda") if fill else torch.zeros(shape, device="cuda")
        if case["cache"] == "same":
            pool[name], pool[name + "_scale"] = x.to(DTYPES[case["dtype"]]).transpose(1, 2), None
        else:
            codes, scale = _quantised(x, case["cache"])
            pool[name], pool[name + "_scale"] = codes.transpose(1, 2), scale.transpose(1, 2)
    return pool, table


def _trees(case, counts, seed):
    """For each sequence which drafted tokens each of them sees: itself and its ancestors in a random tree [B, T, T]."""
    T = case["T"]
    g = torch.Generator().manual_seed(int(seed) + 1)
    sees = torch.zeros((case["B"], T, T), dtype=torch.bool)
    for b in range(case["B"]):
        up = (torch.rand(T, generator=g) * 6).long()
        for t in range(T):
            if t > 0:
                sees[b, t] = sees[b, max(0, t - 1 - int(up[t]))]
            sees[b, t, t] = True
    return sees.cuda()


def prepare(case, seed):
    g = _generator(seed)
    dt = DTYPES[case["dtype"]]
    B, N, D, S = (case[k] for k in ("B", "N", "D", "S"))
    st = {"case": case}
    if case["op"] == "read":
        st["pool"], st["table"] = _pool(case, S, g, True)
        st["lengths"] = _ints(_lengths(case))
        return st
    counts = _counts(case)
    st["counts"] = None if case["counts"] == "all" else _ints(counts)
    T = case["T"]
    if case["op"] == "write":
        st["pool"], st["table"] = _pool(case, S + case["R"], g, S > 0)
        st["start"] = _ints([S - S * (b % 4) // 8 for b in range(B)])
        st["lengths"] = st["start"] + _ints(counts)
        st["key"], st["value"] = (_normal(g, (B, T, N, D), dt) for _ in range(2))
        st["select"] = None
        if case["select"]:  # ascending indices of accepted tokens
            st["select"] = torch.rand((B, T), generator=g, device="cuda").argsort(1)[:, :case["R"]].sort(1)[0].int()
        return st
    st["pool"], st["table"] = _pool(case, S, g, True)
    st["lengths"] = _ints(_lengths(case))
    st["query"] = _normal(g, (B, T, case["M"], D), dt)
    st["key"], st["value"], st["mask"] = None, None, None
    if case["new"] != "none":
        st["key"], st["value"] = (_normal(g, (B, T, N, D), dt) for _ in range(2))
        if case["new"] == "tree":
            st["mask"] = _trees(case, counts, seed)
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _power(e):
    """2^e as float32, exactly (-126 <= e <= 127)."""
    return ((e + 127) << 23).view(torch.float32)


def _quantised(x, how):
    """Codes of the rows of x (float32) and the bytes of their scales: a scale is the least power of two, 2^(byte - 127),
    that brings the row into the codes' range; 255 stands for a row that holds an infinity or a NaN."""
    top = x.abs().amax(-1)
    m, e = torch.frexp(top)
    e = (e.int() - PLACES[how] + (m > MOST[how]).int()).clamp_(min=LEAST)
    e = torch.where(top == 0, LEAST, e)
    fine = torch.isfinite(top)
    scaled = torch.where(fine[..., None], x * _power(torch.where(fine, -e, 0))[..., None], 0.0)
    codes = scaled.to(CODES[how]) if how == "e4m3" else torch.round(scaled).to(CODES[how])
    return codes, torch.where(fine, e + 127, 255).to(torch.uint8)


def _values(codes, scale):
    """What codes with the bytes of their scales stand for, in float32; an unquantised tensor's own values."""
    if scale is None:
        return codes.float()
    s = scale.int()
    return codes.float() * torch.where(s == 255, math.nan, _power(torch.where(s == 255, 0, s - 127)))[..., None]


def _bits(x):
    return x.view(torch.uint8) if x.dtype in (torch.float8_e4m3fn, torch.int8) else x


def _fetch(st, name, rows):
    """The first `rows` tokens of each sequence [B, rows, N, D] in float32."""
    pool, page = st["pool"], st["case"]["page"]
    at = torch.arange(rows, device="cuda")
    block, place = st["table"][:, at // page].long(), at % page
    codes = _bits(pool[name])[block, place].view(pool[name].dtype)
    scale = pool[name + "_scale"]
    return _values(codes, None if scale is None else scale[block, place])


def _plain_read(st):
    case = st["case"]
    rows = case["S"] if case["op"] == "read" else case["S"] + case["R"]
    here = (torch.arange(rows, device="cuda") < st["lengths"][:, None])[..., None, None]
    dt = DTYPES[case["dtype"]]
    return {n: torch.where(here, _fetch(st, n, rows), 0.0).to(dt) for n in ("key", "value")}


def _plain_write(st):
    case, pool, page = st["case"], st["pool"], st["case"]["page"]
    B, R = case["B"], case["R"]
    r = torch.arange(R, device="cuda")
    at = (st["start"][:, None] + r).long()
    block, place = st["table"].gather(1, at // page).long(), at % page
    if st["counts"] is not None:
        here = r < st["counts"][:, None]
        block, place = block[here], place[here]
    for name in ("key", "value"):
        x = st[name]
        if st["select"] is not None:
            x = x[torch.arange(B, device="cuda")[:, None], st["select"].long()]
        if st["counts"] is not None:
            x = x[here]
        if case["cache"] == "same":
            pool[name][block, place] = x
        else:
            codes, scale = _quantised(x.float(), case["cache"])
            _bits(pool[name])[block, place] = _bits(codes)
            pool[name + "_scale"][block, place] = scale
    if case["cache"] == "same":
        return {"key": pool["key"], "value": pool["value"]}
    return _plain_read(st)


def _plain_attention(st):
    case = st["case"]
    B, T, S, M, N, D = (case[k] for k in ("B", "T", "S", "M", "N", "D"))
    dt = DTYPES[case["dtype"]]
    k, v = _fetch(st, "key", S), _fetch(st, "value", S)
    seen = (torch.arange(S, device="cuda") < st["lengths"][:, None])[:, None].expand(B, T, S)
    t = torch.arange(T, device="cuda")
    if case["new"] != "none":
        k, v = torch.cat((k, st["key"].float()), 1), torch.cat((v, st["value"].float()), 1)
        mine = st["mask"] if case["new"] == "tree" else (t[None, :] <= t[:, None])[None].expand(B, T, T)
        if st["counts"] is not None:
            mine = mine & (t < st["counts"][:, None])[:, None]
        seen = torch.cat((seen, mine), 2)
    if st["counts"] is not None:
        seen = seen & (t < st["counts"][:, None])[..., None]
    q = st["query"].float().view(B, T, N, M // N, D).permute(0, 2, 3, 1, 4).reshape(B, N, -1, D)   # [B, N, G T, D]
    s = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(1.0 / math.sqrt(D)).view(B, N, M // N, T, -1)
    s.masked_fill_(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total))[..., 0].reshape(B, M, T)
    p.div_(torch.where(total == 0, torch.ones_like(total), total))
    o = torch.matmul(p.view(B, N, (M // N) * T, -1), v.permute(0, 2, 1, 3)).view(B, N, M // N, T, D)
    return {"out": o.permute(0, 3, 1, 2, 4).reshape(B, T, M * D).to(dt), "lse": lse}


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _own_run(st):
    import scale_deformable_attention_gb300 as msda

    case = st["case"]
    cache = msda.PagedCache(**st["pool"])
    dt = DTYPES[case["dtype"]]
    if case["op"] == "attention":
        out, lse = msda.cache_attention(st["query"], cache, st["table"], st["lengths"], st["key"], st["value"],
                                        mask=st["mask"], counts=st["counts"])
        return {"out": out, "lse": lse}
    if case["op"] == "read":
        key, value = msda.cache_read(cache, st["table"], st["lengths"], case["S"], dtype=dt)
        return {"key": key, "value": value}
    msda.cache_write(cache, st["key"], st["value"], st["table"], st["start"], counts=st["counts"],
                     select=st["select"])
    if case["cache"] == "same":
        return {"key": cache.key, "value": cache.value}
    key, value = msda.cache_read(cache, st["table"], st["lengths"], case["S"] + case["R"], dtype=dt)
    return {"key": key, "value": value}


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    return _plain_attention(state) if op == "attention" else _plain_read(state) if op == "read" else _plain_write(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    N, D, B = case["N"], case["D"], case["B"]
    row = N * D * es * 2                                              # a token's key and value
    kept = row if case["cache"] == "same" else N * (D + 1) * 2        # the same in the cache
    if case["op"] == "read":
        n = sum(_lengths(case))
        return {"bytes": n * kept + B * case["S"] * row, "flops": n * N * D * 2}
    counts = _counts(case)
    if case["op"] == "write":
        n = sum(counts)
        moved, flops = n * (row + kept), 0
        if case["cache"] != "same":                                   # read back
            all_rows = n + sum(case["S"] - case["S"] * (b % 4) // 8 for b in range(B))
            moved += all_rows * kept + B * (case["S"] + case["R"]) * row
            flops = (n + all_rows) * N * D * 2
        return {"bytes": moved, "flops": flops}
    T, M = case["T"], case["M"]
    lengths = _lengths(case)
    pairs = sum(n * c for n, c in zip(lengths, counts))
    moved = sum(lengths) * kept + B * T * M * (D * es * 2 + 4)
    if case["new"] != "none":
        moved += sum(counts) * row
        moved += B * T * T if case["new"] == "tree" else 0
        pairs += sum(c * (c + 1) // 2 if case["new"] == "chain" else c * min(c, 6) for c in counts)
    return {"bytes": moved, "flops": pairs * M * D * 4}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _two_to(e):
    """2^e in 64 bits for whole e, put together from its bits (a power function may be off in the last place)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_values(codes, scale):
    if scale is None:
        return codes.double()
    s = _two_to(scale.long() - 127)
    s[scale == 255] = math.nan
    return codes.double() * s[..., None]


def _exact_code(x, how):
    """The values that x's rows are held as: the nearest of the codes' values times the scale, ties to the even code."""
    x = x.double()
    top = x.abs().max(-1, keepdim=True)[0]
    most = 448.0 if how == "e4m3" else 127.0
    e = torch.ceil(torch.log2(torch.where(top > 0, top, 1.0) / most))
    e = torch.where(top > most * _two_to(e), e + 1, e)                # the logarithm is rounded
    e = torch.where(top <= most * _two_to(e - 1), e - 1, e)
    scale = _two_to(torch.where(top > 0, e.clamp(min=-100.0), -100.0))
    y = x / scale
    if how == "int8":
        return torch.round(y) * scale
    step = _two_to(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)  # three binary places behind the first, 2^-9 at least
    return torch.round(y / step) * step * scale


def _exact_rows(st, b, name, rows):
    page, pool = st["case"]["page"], st["pool"]
    at = torch.arange(rows, device="cuda")
    block = st["table"][b].long()[torch.div(at, page, rounding_mode="floor")]
    codes = _bits(pool[name])[block, at % page].view(pool[name].dtype)
    scale = pool[name + "_scale"]
    return _exact_values(codes, None if scale is None else scale[block, at % page])


def _exact_write(case, st):
    counts = _counts(case)
    got = {}
    for name in ("key", "value"):
        pool = st["pool"][name].double() if case["cache"] == "same" else None
        kept = torch.zeros((case["B"], case["S"] + case["R"], case["N"], case["D"]), dtype=torch.float64, device="cuda")
        for b in range(case["B"]):
            first, n = int(st["start"][b]), counts[b]
            x = st[name][b] if st["select"] is None else st[name][b][st["select"][b].long()]
            at = torch.arange(first, first + n, device="cuda")
            if case["cache"] == "same":
                pool[st["table"][b].long()[at // case["page"]], at % case["page"]] = x[:n].double()
            else:
                kept[b, :first] = _exact_rows(st, b, name, first)
                kept[b, first:first + n] = _exact_code(x[:n], case["cache"])
        got[name] = kept if pool is None else pool
    return got


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "write":
        return _exact_write(case, st)
    B, S, N, D = (case[k] for k in ("B", "S", "N", "D"))
    dev = {"dtype": torch.float64, "device": "cuda"}
    lengths = _lengths(case)
    if case["op"] == "read":
        got = {n: torch.zeros((B, S, N, D), **dev) for n in ("key", "value")}
        for b in range(B):
            for name in got:
                got[name][b, :lengths[b]] = _exact_rows(st, b, name, lengths[b])
        return got
    T, M = case["T"], case["M"]
    counts = _counts(case)
    out, lse = torch.zeros((B, T, M, D), **dev), torch.full((B, M, T), -math.inf, **dev)
    for b in range(B):
        c = counts[b]
        keys, values = _exact_rows(st, b, "key", lengths[b]), _exact_rows(st, b, "value", lengths[b])
        hidden = torch.zeros((c, lengths[b]), dtype=torch.bool, device="cuda")
        if case["new"] != "none":
            keys = torch.cat((keys, st["key"][b, :c].double()))
            values = torch.cat((values, st["value"][b, :c].double()))
            mine = torch.tril(torch.ones((c, c), dtype=torch.bool, device="cuda"))
            if case["new"] == "tree":
                mine = st["mask"][b, :c, :c]
            hidden = torch.cat((hidden, ~mine), 1)
        if keys.shape[0] == 0:
            continue
        for m in range(M):
            n = m // (M // N)
            s = st["query"][b, :c, m].double() @ keys[:, n].T * D ** -0.5
            s[hidden] = -math.inf
            z = torch.logsumexp(s, -1, keepdim=True)
            p = torch.exp(s - torch.where(z == -math.inf, 0.0, z))
            out[b, :c, m], lse[b, m, :c] = p @ values[:, n], z[:, 0]
    return {"out": out.view(B, T, M * D), "lse": lse}
