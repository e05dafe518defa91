"""Dense softmax attention and its gradients on the GPU against the definition
in 64 bits, with bounds worked out from the inputs (dense_reference)."""
import math

import pytest

import dense_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def msda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import scale_deformable_attention_gb300 as m

    yield m
    assert m.device_errors() == 0


def make(seed, dtype, B, Q, S, M, N, D):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device=DEV).to(DT[dtype])   # noqa: E731
    return n(B, Q, M, D), n(B, S, N, D), n(B, S, N, D), n(B, Q, M * D)


def masks(kind, seed, B, Q, S, M):
    """(keyword arguments, allowed pairs)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s: torch.rand(s, generator=g, device=DEV)                 # noqa: E731
    kw, ok = {}, None
    if "keys" in kind:
        km = rnd(B, S) < 0.7
        if "none" in kind:
            km[0] = False
        kw["key_mask"] = km
        ok = km[:, None, None, :]
    if "pairs" in kind:
        shape = (B, M, Q, S) if "each" in kind else (Q, S)
        m = rnd(*shape) < 0.6
        m[..., Q // 2, :] = False                    # a row that sees nothing
        if S > 2:
            m[..., S // 3] = False                   # a key that nobody sees
        kw["mask"] = m
        mm = m if m.dim() == 4 else m[None, None]
        ok = mm if ok is None else ok & mm
    if "causal" in kind:
        kw["causal"] = True
        i = torch.arange(Q, device=DEV)[:, None] + (S - Q)
        c = (torch.arange(S, device=DEV)[None] <= i)[None, None]
        ok = c if ok is None else ok & c
    return kw, ok


def both(msda, q, k, v, do, kw):
    out, lse = msda.attention_forward(q, k, v, **kw)
    gq, gk, gv = msda.attention_backward(q, k, v, out, lse, do, **kw)
    return {"out": out, "lse": lse, "grad_query": gq, "grad_key": gk, "grad_value": gv}


SIZES = [
    # B, Q, S, M, N, D
    (1, 1, 1, 1, 1, 32), (2, 5, 3, 2, 2, 8), (1, 128, 128, 1, 1, 64), (2, 127, 129, 4, 2, 32), (1, 257, 130, 2, 1, 128),
    (3, 1, 700, 8, 2, 64), (1, 300, 300, 8, 8, 32), (2, 64, 511, 6, 2, 48), (1, 200, 513, 3, 1, 96),
    (1, 130, 260, 7, 1, 80), (2, 33, 65, 2, 2, 20), (1, 70, 90, 2, 1, 7), (1, 1, 5000, 16, 1, 128),
    (1, 1000, 1, 2, 2, 16), (1, 640, 385, 2, 2, 112), (9, 17, 31, 1, 1, 24), (1, 389, 1025, 5, 5, 40),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_sizes(msda, size, dtype):
    q, k, v, do = make(1, dtype, *size)
    want = R.attention(q, k, v, do)
    got = both(msda, q, k, v, do, {})
    for name in want:
        R.check(got[name], want[name], name)


MASKED = [(2, 127, 129, 4, 2, 32), (1, 257, 130, 2, 1, 128), (3, 1, 700, 8, 2, 64), (2, 300, 300, 2, 2, 32),
          (2, 130, 700, 3, 1, 64), (1, 400, 130, 2, 2, 48), (2, 33, 65, 2, 2, 20)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind", ["keys", "keys none", "pairs", "pairs each", "causal", "keys pairs", "keys causal",
                                  "keys pairs each causal"])
@pytest.mark.parametrize("size", MASKED, ids=lambda s: "x".join(map(str, s)))
def test_masks(msda, size, kind, dtype):
    B, Q, S, M, N, D = size
    q, k, v, do = make(2, dtype, *size)
    kw, ok = masks(kind, 3, B, Q, S, M)
    want = R.attention(q, k, v, do, ok)
    got = both(msda, q, k, v, do, kw)
    for name in want:
        R.check(got[name], want[name], name)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("kind", ["", "keys none", "pairs", "pairs each", "causal"])
@pytest.mark.parametrize("size", [(20, 300, 260, 8, 8, 32), (10, 513, 140, 16, 16, 128), (30, 300, 300, 6, 6, 80),
                                  (20, 70, 400, 24, 8, 64)], ids=lambda s: "x".join(map(str, s)))
def test_many_rows(msda, size, kind, dtype):
    """Enough rows for every SM to take two row tiles at a time."""
    B, Q, S, M, N, D = size
    q, k, v, do = make(19, dtype, *size)
    kw, ok = masks(kind, 20, B, Q, S, M)
    want = R.attention(q, k, v, do, ok)
    got = both(msda, q, k, v, do, kw)
    for name in want:
        R.check(got[name], want[name], name)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind", ["keys", "pairs", "keys pairs"])
@pytest.mark.parametrize("D", [32, 128, 20])
def test_masked_places_may_hold_anything(msda, kind, dtype, D):
    """Keys and values that no query sees, and queries and gradients of rows without keys, hold NaN and infinity."""
    B, Q, S, M, N = 2, 150, 300, 4, 2
    q, k, v, do = make(4, dtype, B, Q, S, M, N, D)
    kw, ok = masks(kind, 5, B, Q, S, M)
    want = R.attention(q, k, v, do, ok)
    seen = ok.expand(B, M, Q, S).reshape(B, N, M // N, Q, S).any(3).any(2).transpose(1, 2)      # [B, S, N]
    bad = torch.where(torch.arange(S, device=DEV) % 2 == 0, math.nan, math.inf)[None, :, None, None].to(k.dtype)
    k = torch.where(seen[..., None], k, bad)
    v = torch.where(seen[..., None], v, bad)
    empty = ~ok.expand(B, M, Q, S).any(-1).transpose(1, 2)                                       # [B, Q, M]
    q = torch.where(empty[..., None], torch.full_like(q, math.nan), q)
    do = torch.where(empty[..., None], torch.full_like(q, math.inf), do.view(B, Q, M, D)).reshape(B, Q, M * D)
    got = both(msda, q, k, v, do, kw)
    for name in want:
        R.check(got[name], want[name], name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("how", ["fused", "heads first", "expanded", "misaligned", "reversed channels"])
def test_strides(msda, how, dtype):
    B, Q, M, D = 2, 150, 4, 32
    q, k, v, do = make(6, dtype, B, Q, Q, M, M, D)
    if how == "fused":                # one projection's output
        x = torch.cat((q, k, v), 2).contiguous()
        q, k, v = x[:, :, :M], x[:, :, M:2 * M], x[:, :, 2 * M:]
    elif how == "heads first":        # [B, M, Q, D] storage
        q, k, v = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k, v))
    elif how == "expanded":           # one image's keys for both
        k, v = k[:1].expand(B, -1, -1, -1), v[:1].expand(B, -1, -1, -1)
    elif how == "misaligned":
        shift = lambda t: torch.cat((t.reshape(-1)[:1], t.reshape(-1)))[1:].view(t.shape)   # noqa: E731
        q, k, v = shift(q), shift(k), shift(v)
    else:
        q = q.transpose(2, 3).contiguous().transpose(2, 3)
    want = R.attention(q, k, v, do)
    got = both(msda, q, k, v, do, {})
    for name in want:
        R.check(got[name], want[name], name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 300), (2, 1, 1, 300), (4, 1, 300), (1, 4, 70, 300), (2, 1, 70, 300), (70, 300)])
def test_broadcast_masks(msda, shape, dtype):
    B, Q, S, M, N, D = 2, 70, 300, 4, 2, 64
    q, k, v, do = make(21, dtype, B, Q, S, M, N, D)
    mask = torch.rand(shape, device=DEV, generator=torch.Generator(device=DEV).manual_seed(22)) < 0.5
    want = R.attention(q, k, v, do, mask.view((1,) * (4 - mask.dim()) + tuple(shape)))
    for m in (mask, torch.stack((mask, ~mask), -1)[..., 0]):      # the second: keys are not next to one another
        got = both(msda, q, k, v, do, {"mask": m})
        for name in want:
            R.check(got[name], want[name], name)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size", [(1, 37, 200, 16, 1, 32), (2, 3, 1500, 32, 2, 64), (1, 150, 140, 9, 1, 128),
                                  (1, 2, 300, 130, 1, 16), (300, 5, 6, 2, 1, 24)], ids=lambda s: "x".join(map(str, s)))
def test_shared_heads(msda, size, dtype):
    """Few and many query heads on one key head, more than a row tile holds, and many batch items."""
    B, Q, S, M, N, D = size
    q, k, v, do = make(23, dtype, *size)
    kw, ok = masks("keys causal", 24, B, Q, S, M)
    want = R.attention(q, k, v, do, ok)
    got = both(msda, q, k, v, do, kw)
    for name in want:
        R.check(got[name], want[name], name)


@pytest.mark.parametrize("dtype,D", [("f32", 48), ("bf16", 64), ("bf16", 72), ("f16", 20)])
def test_nothing_is_written_outside(msda, dtype, D):
    """Outputs inside larger buffers: what lies before and behind them stays (sizes that end inside every tile)."""
    from scale_deformable_attention_gb300 import _lib
    from scale_deformable_attention_gb300._attention import _problem

    B, Q, S, M, N = 2, 131, 197, 4, 2
    q, k, v, do = make(25, dtype, B, Q, S, M, N, D)
    _, _, _, _, _, flags, p, scale, _ = _problem(q, k, v, None, None, True, None)
    lib, dt = _lib.lib(), {"f32": 0, "f16": 1, "bf16": 2}[dtype]
    pad = 1024

    def guarded(n, t):
        buf = torch.full((n + 2 * pad,), -7.0, dtype=t, device=DEV)
        return buf, buf[pad:pad + n]

    st = torch.cuda.current_stream().cuda_stream
    need = max(lib.msda_attention_forward_workspace_size(dt, flags, p), lib.msda_attention_backward_workspace_size(dt, flags, p))
    wb = torch.full((need + 4096,), 77, dtype=torch.uint8, device=DEV)
    bufs = {n: guarded(e, t) for n, e, t in (("out", q.numel(), q.dtype), ("lse", B * M * Q, torch.float32),
                                             ("gq", q.numel(), q.dtype), ("gk", k.numel(), q.dtype), ("gv", v.numel(), q.dtype))}
    ptr = {n: b[1].data_ptr() for n, b in bufs.items()}
    _lib.check(lib.msda_attention_forward(dt, flags, p, scale, q.data_ptr(), k.data_ptr(), v.data_ptr(), None, None,
                                          ptr["out"], ptr["lse"], wb.data_ptr(), need, st))
    _lib.check(lib.msda_attention_backward(dt, flags, p, scale, q.data_ptr(), k.data_ptr(), v.data_ptr(), None, None,
                                           ptr["out"], ptr["lse"], do.data_ptr(), ptr["gq"], ptr["gk"], ptr["gv"],
                                           wb.data_ptr(), need, st))
    torch.cuda.synchronize()
    for name, (buf, inner) in bufs.items():
        assert (buf[:pad] == -7).all() and (buf[-pad:] == -7).all(), name
        assert torch.isfinite(inner.float()).all() or name == "lse", name
    assert (wb[need:] == 77).all()
    want = both(msda, q, k, v, do, {"causal": True})
    for a, b in (("out", "out"), ("lse", "lse"), ("gq", "grad_query"), ("gk", "grad_key"), ("gv", "grad_value")):
        assert torch.equal(bufs[a][1], want[b].reshape(-1)), a


def test_two_calls_at_once(msda):
    """Two streams at the same time, forward and gradients, many times: each gives the lone call's bits."""
    size = (2, 500, 900, 8, 4, 64)
    ins = [make(s, "bf16", *size) for s in (26, 27)]
    kw, _ = masks("pairs", 28, 2, 500, 900, 8)
    alone = [both(msda, *t, kw) for t in ins]
    streams = [torch.cuda.Stream() for _ in ins]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for st, t in zip(streams, ins):
            with torch.cuda.stream(st):
                got.append(both(msda, *t, kw))
        torch.cuda.synchronize()
        for a, g in zip(alone, got):
            for name in a:
                assert torch.equal(a[name], g[name]), name


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_large_scores_and_gradients(msda, dtype):
    """Scores far apart (one key takes everything) and gradients of a scaled loss."""
    B, Q, S, M, N, D = 1, 140, 270, 2, 1, 64
    q, k, v, do = make(7, dtype, B, Q, S, M, N, D)
    q = q * 6
    do = (do.float() * 200).to(do.dtype)
    want = R.attention(q, k, v, do)
    got = both(msda, q, k, v, do, {})
    for name in want:
        R.check(got[name], want[name], name)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_rising_scores(msda, dtype):
    """Every tile's maximum is above the one before: each forces the running output to be rescaled."""
    B, Q, S, M, D = 1, 130, 1000, 2, 32
    q, k, v, do = make(8, dtype, B, Q, S, M, M, D)
    q = q.abs()
    k = (k.float().abs() * (torch.arange(S, device=DEV) / 200.0)[None, :, None, None]).to(k.dtype)
    want = R.attention(q, k, v, do)
    got = both(msda, q, k, v, do, {})
    for name in want:
        R.check(got[name], want[name], name)


def test_small_values_in_half_precision(msda):
    """Long rows of even probabilities: p and ds are below binary16's normal range."""
    B, Q, S, M, D = 1, 64, 20000, 1, 32
    q, k, v, do = make(9, "f16", B, Q, S, M, M, D)
    want = R.attention(q, k, v, do)
    got = both(msda, q, k, v, do, {})
    for name in want:
        R.check(got[name], want[name], name)
        value = want[name][0]
        rel = float((got[name].double().reshape(value.shape) - value).norm() / value.norm())
        # three independent roundings of at most half a step, uniform: sqrt(3) * 2^-11 / sqrt(3), twice that as the limit
        assert rel <= 2 * 2.0 ** -11, (name, rel)


@pytest.mark.parametrize("S", [2, 3, 7, 40, 128])
def test_few_keys_keep_their_gradients(msda, S):
    """With few keys the output is as large as a value: delta = <dout, out> from its 16 bits would carry an error of
    |dout| |out| 2^-8 into differences dP - delta that are smaller.  Left are the roundings of dS, of P and of the result, each
    uniform within 2^-8 (2^-8 / sqrt(3) of a value in the root mean square): at most 2^-8 together."""
    for D in (8, 96):
        q, k, v, do = make(29, "bf16", 7, 3, S, 16, 16, D)
        want = R.attention(q, k, v, do)
        got = both(msda, q, k, v, do, {})
        for name in ("grad_query", "grad_key", "grad_value"):
            value = want[name][0]
            assert float((got[name].double() - value).norm() / value.norm()) <= 2.0 ** -8, (name, D)


def test_empty_tensors(msda):
    dev = torch.device(DEV)
    for B, Q, S in ((0, 5, 5), (2, 0, 5), (2, 5, 0), (0, 0, 0)):
        q = torch.randn(B, Q, 2, 32, device=dev, dtype=torch.bfloat16)
        k = torch.randn(B, S, 2, 32, device=dev, dtype=torch.bfloat16)
        out, lse = msda.attention_forward(q, k, k)
        assert out.shape == (B, Q, 64) and lse.shape == (B, 2, Q)
        assert not out.any() and (lse == -math.inf).all()
        got = msda.attention_backward(q, k, k, out, lse, torch.ones_like(out))
        assert [tuple(g.shape) for g in got] == [tuple(q.shape), tuple(k.shape), tuple(k.shape)]
        assert not any(g.any() for g in got)


@pytest.mark.parametrize("dtype,D", [("f32", 48), ("bf16", 64), ("f16", 32), ("bf16", 128)])
def test_same_bits_every_run(msda, dtype, D):
    q, k, v, do = make(10, dtype, 2, 700, 900, 4, 2, D)
    one = both(msda, q, k, v, do, {"causal": True})
    for _ in range(3):
        two = both(msda, q, k, v, do, {"causal": True})
        for name in one:
            assert torch.equal(one[name], two[name]), name


@pytest.mark.parametrize("dtype,size", [("bf16", (2, 300, 300, 8, 2, 32)), ("f32", (1, 100, 200, 2, 2, 48)),
                                        ("f16", (2, 1, 3000, 8, 2, 64))])
def test_autograd_and_differences(msda, dtype, size):
    """The operator's gradients are the formula's, and the 64-bit loss moves by them."""
    B, Q, S, M, N, D = size
    q, k, v, do = make(11, dtype, *size)
    kw, ok = masks("keys", 12, B, Q, S, M)
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    out = msda.attention(*leaves, **kw)
    assert out.shape == (B, Q, M * D)
    got = torch.autograd.grad(out, leaves, do)
    want = R.attention(q, k, v, do, ok)
    for g, name in zip(got, ("grad_query", "grad_key", "grad_value")):
        R.check(g, want[name], name)
    # central differences of the definition along a random direction, in 64 bits: off by h^2 times the third
    # derivative; h = 1e-4 leaves 1e-6 of the sum of sizes
    loss = lambda a, b, c: (R.attention(a, b, c, None, ok)["out"][0] * do.double()).sum()    # noqa: E731
    h = 1e-4
    for i, g in enumerate(got):
        d = torch.randn_like(leaves[i], dtype=torch.float64)
        base = [t.detach().double() for t in leaves]
        plus, minus = list(base), list(base)
        plus[i], minus[i] = base[i] + h * d, base[i] - h * d
        num = float((loss(*plus) - loss(*minus)) / (2 * h))
        name = ("grad_query", "grad_key", "grad_value")[i]
        limit = float((want[name][1] * d.abs()).sum()) + 1e-6 * float((want[name][0] * d).abs().sum())
        assert abs(float((g.double() * d).sum()) - num) <= limit


def test_graph_replay_and_side_stream(msda):
    """Captured forward and backward, replayed on other inputs, give an eager call's bits; so does another stream."""
    size = (2, 300, 700, 4, 2, 64)
    q, k, v, do = make(13, "bf16", *size)
    kw, _ = masks("keys pairs", 14, 2, 300, 700, 4)
    both(msda, q, k, v, do, kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = both(msda, q, k, v, do, kw)
    torch.cuda.current_stream().wait_stream(s)
    here = both(msda, q, k, v, do, kw)
    torch.cuda.synchronize()
    for name in here:
        assert torch.equal(here[name], side[name]), name
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        one = both(msda, q, k, v, do, kw)
    with torch.cuda.graph(g2):
        two = both(msda, q, k, v, do, kw)
    fresh = make(15, "bf16", *size)
    for t, f in zip((q, k, v, do), fresh):
        t.copy_(f)
    g1.replay()
    g2.replay()
    torch.cuda.synchronize()
    eager = both(msda, q, k, v, do, kw)
    for name in eager:
        assert torch.equal(eager[name], one[name]) and torch.equal(eager[name], two[name]), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_past_32_bits(msda, dtype):
    """Batch items more than 2^31 elements apart."""
    B, Q, S, M, D = 2, 3, 200, 1, 32
    far = 2 ** 31 + 64
    q, k, v, do = make(16, dtype, B, Q, S, M, M, D)
    want = R.attention(q, k, v, do)
    store = torch.empty(far + S * D, dtype=k.dtype, device=DEV)
    kk = store.as_strided((B, S, M, D), (far, D, D, 1))
    kk.copy_(k)
    got = both(msda, q, kk, v, do, {})
    for name in want:
        R.check(got[name], want[name], name)
    del store, kk
    torch.cuda.empty_cache()


def test_with_the_sampled_attention(msda):
    """A decoder layer's core: norm and rotation of queries and keys, attention among the queries, sampled attention."""
    B, Q, M, D, L, K = 2, 100, 4, 32, 2, 4
    g = torch.Generator(device=DEV).manual_seed(17)
    bf = torch.bfloat16
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV)                # noqa: E731
    shapes = torch.tensor([(20, 30), (10, 15)], device=DEV)
    S = 20 * 30 + 10 * 15
    x = rnd(B, Q, 3 * M, D).to(bf).requires_grad_()
    w = [(1 + 0.1 * rnd(D)).to(bf).requires_grad_() for _ in range(2)]
    ref = torch.rand((B, Q, 2), generator=g, device=DEV)
    freq = 100.0 ** (-torch.arange(8, device=DEV) / 8.0)
    freq = torch.cat((freq, freq)).float()
    value = rnd(B, S, M, D).to(bf).requires_grad_()
    attn = torch.softmax(rnd(B, Q, M, L * K), -1).view(B, Q, M, L, K).to(bf)
    base = torch.rand((B, Q, M, L, K, 2), generator=g, device=DEV).to(bf)
    do = rnd(B, Q, M * D).to(bf)

    def layer():
        q, k = msda.norm_rotary(x[:, :, :M], x[:, :, M:2 * M], w[0], w[1], ref * 32, freq, (8, 8))
        a = msda.attention(q, k, x[:, :, 2 * M:])
        loc = base + 0.01 * a.view(B, Q, M, D)[..., :16].reshape(B, Q, M, L, K, 2)
        return msda.multi_scale_deformable_attention(value, shapes, None, loc, attn), q, k, a

    out, q, k, a = layer()
    grads = torch.autograd.grad(out, [x, value, *w], do)
    n = [R.norm_rotary(t, wt, ref * 32, freq, (8, 8), False, 1e-6)["out"]
         for t, wt in ((x[:, :, :M], w[0]), (x[:, :, M:2 * M], w[1]))]
    R.check(q, n[0], "query")
    R.check(k, n[1], "key")
    R.check(a, R.attention(q.detach(), k.detach(), x[:, :, 2 * M:].detach())["out"], "attention")
    assert all(t.shape == s.shape and torch.isfinite(t).all() and t.any() for t, s in zip(grads, [x, value, *w]))


def test_refusals(msda):
    q, k, v, do = make(18, "bf16", 1, 4, 6, 4, 2, 32)
    with pytest.raises(ValueError):
        msda.attention_forward(q[0], k, v)
    with pytest.raises(ValueError):
        msda.attention_forward(q, k, v[:, :5])
    with pytest.raises(TypeError):
        msda.attention_forward(q, k.float(), v)
    with pytest.raises(ValueError):
        msda.attention_forward(q[:, :, :3], k, v)
    with pytest.raises(ValueError):
        msda.attention_forward(q.cpu(), k.cpu(), v.cpu())
    with pytest.raises(TypeError):
        msda.attention_forward(q, k, v, mask=torch.zeros(4, 6, device=DEV))
    with pytest.raises(ValueError):
        msda.attention_forward(q, k, v, mask=torch.ones(5, 6, dtype=torch.bool, device=DEV))
    with pytest.raises(ValueError):
        msda.attention_forward(q, k, v, key_mask=torch.ones(2, 6, dtype=torch.bool, device=DEV))
    with pytest.raises(ValueError):
        msda.attention_forward(q, k, v, mask=torch.ones(4, 6, dtype=torch.bool))
    with pytest.raises(msda.MsdaError):
        msda.attention_forward(q, k, v, scale=-1.0)
    wide = torch.zeros(1, 4, 2, 136, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(msda.MsdaError):
        msda.attention_forward(wide, wide, wide)
    out, lse = msda.attention_forward(q, k, v)
    with pytest.raises(ValueError):
        msda.attention_backward(q, k, v, out, lse.double(), do)
    with pytest.raises(ValueError):
        msda.attention_backward(q, k, v, out, lse, do.float())
    many = torch.zeros(1, 4000, 2, 32, dtype=torch.float32, device=DEV)
    with pytest.raises(msda.MsdaError):
        msda.attention_forward(many[:, :1], many, many, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
