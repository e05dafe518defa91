"""Rotary positions with several axes and the norm with rotation on the GPU
against the definition in 64 bits, with bounds worked out from the inputs."""
import math

import pytest

import dense_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


@pytest.fixture(scope="module")
def msda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import scale_deformable_attention_gb300 as m

    return m


def make(seed, dtype, B, S, heads, D):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [torch.randn((B, S, h, D), generator=g, device=DEV).to(DT[dtype]) for h in heads]


def how(kind, B, S, sections, seed=0):
    g = torch.Generator(device=DEV).manual_seed(100 + seed)
    A = len(sections)
    if kind == "float":
        pos = torch.rand((B, S, A), generator=g, device=DEV) * 1333
    else:
        start = {"int": 0, "far": 16_700_000, "beyond": 2 ** 33}[kind]
        pos = torch.randint(0, 4000, (1 if kind == "int" else B, S, A), generator=g, device=DEV) + start
        if kind == "int":
            pos = pos.int()
    f = [1000.0 ** (-j / n) for n in sections for j in range(n)]
    return pos, torch.tensor(f, dtype=torch.float32, device=DEV), sections


CASES = [
    # B, S, M, N, D, sections, positions
    (1, 1, 1, 1, 32, (8, 8), "float"), (2, 37, 8, 8, 32, (8, 8), "float"), (1, 300, 8, 2, 64, (12, 10, 10), "int"),
    (3, 65, 5, 1, 48, (12, 12), "far"), (1, 130, 16, 4, 128, (16, 24, 16), "beyond"), (2, 33, 2, 2, 20, (5, 3), "float"),
    (1, 9, 3, 3, 7, (2,), "int"), (1, 700, 1, 1, 256, (64, 32, 16, 16), "far"), (2, 50, 4, 1, 96, (24, 0, 24), "int"),
    (1, 64, 40, 3, 16, (8,), "float"), (2, 11, 2, 1, 8, (0, 0), "float"), (1, 2000, 8, 8, 80, (20, 12), "float"),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[:5])))
def test_norm_rotary(msda, case, interleaved, dtype):
    B, S, M, N, D, sections, kind = case
    q, k, gq, gk = make(1, dtype, B, S, (M, N, M, N), D)
    wq, wk = (1 + 0.2 * torch.randn((2, D), device=DEV, generator=torch.Generator(device=DEV).manual_seed(2))).to(q.dtype)
    h = how(kind, B, S, sections)
    oq, ok = msda.norm_rotary_forward(q, k, wq, wk, *h, eps=EPS, interleaved=interleaved)
    got = msda.norm_rotary_backward(q, k, wq, wk, *h, gq, gk, eps=EPS, interleaved=interleaved)
    again = msda.norm_rotary_backward(q, k, wq, wk, *h, gq, gk, eps=EPS, interleaved=interleaved)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    for x, w, g, out, dx, dw in ((q, wq, gq, oq, got[0], got[2]), (k, wk, gk, ok, got[1], got[3])):
        want = R.norm_rotary(x, w, *h, interleaved, EPS, g)
        R.check(out, want["out"], "out")
        R.check(dx, want["grad"], "grad")
        R.check(dw, want["grad_weight"], "grad_weight")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[:5])))
def test_rotary(msda, case, interleaved, dtype):
    B, S, M, N, D, sections, kind = case
    x, g = make(3, dtype, B, S, (M, M), D)
    h = how(kind, B, S, sections)
    want = R.norm_rotary(x, None, *h, interleaved, EPS, g)
    R.check(msda.rotary_forward(x, *h, interleaved=interleaved), want["out"], "out")
    R.check(msda.rotary_backward(g, *h, interleaved=interleaved), want["grad"], "grad")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["fused", "heads first", "misaligned", "expanded", "channels apart"])
def test_strides(msda, layout, dtype):
    B, S, M, N, D = 2, 70, 4, 2, 32
    q, k, gq, gk = make(4, dtype, B, S, (M, N, M, N), D)
    if layout == "fused":
        x = torch.cat((q, k), 2).contiguous()
        q, k = x[:, :, :M], x[:, :, M:]
    elif layout == "heads first":
        q, k, gq = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k, gq))
    elif layout == "misaligned":
        q, k, gk = (torch.cat((t.reshape(-1)[:1], t.reshape(-1)))[1:].view(t.shape) for t in (q, k, gk))
    elif layout == "expanded":
        k, gk = k[:1].expand(B, -1, -1, -1), gk[:, :, :1].expand(-1, -1, N, -1)
    else:
        q = q.transpose(2, 3).contiguous().transpose(2, 3)
    wq, wk = torch.ones((2, D), device=DEV, dtype=q.dtype)
    h = how("float", B, S, (8, 8))
    oq, ok = msda.norm_rotary_forward(q, k, wq, wk, *h)
    got = msda.norm_rotary_backward(q, k, wq, wk, *h, gq, gk)
    for x, w, g, out, dx, dw in ((q, wq, gq, oq, got[0], got[2]), (k, wk, gk, ok, got[1], got[3])):
        want = R.norm_rotary(x, w, *h, False, EPS, g)
        R.check(out, want["out"], "out")
        R.check(dx, want["grad"], "grad")
        R.check(dw, want["grad_weight"], "grad_weight")


def test_large_and_zero_rows(msda):
    """Rows of zeros keep eps under the root; rows of large values do not overflow binary32."""
    q, k = make(5, "bf16", 1, 40, (4, 4), 64)
    q[:, 3] = 0
    k[:, 5] = k[:, 5] * 2.0 ** 40
    w = torch.ones(64, device=DEV, dtype=q.dtype)
    h = how("float", 1, 40, (16, 16))
    oq, ok = msda.norm_rotary_forward(q, k, w, w, *h)
    for x, out in ((q, oq), (k, ok)):
        R.check(out, R.norm_rotary(x, w, *h, False, EPS)["out"], "out")
    assert not oq[:, 3].any()


def test_autograd_and_differences(msda):
    B, S, M, N, D = 2, 21, 3, 1, 32
    q, k, gq, gk = make(6, "f32", B, S, (M, N, M, N), D)
    wq, wk = 1 + 0.2 * torch.randn((2, D), device=DEV, generator=torch.Generator(device=DEV).manual_seed(7))
    h = how("float", B, S, (8, 8))
    leaves = [t.clone().requires_grad_() for t in (q, k, wq, wk)]
    oq, ok = msda.norm_rotary(*leaves, *h)
    got = torch.autograd.grad((oq, ok), leaves, (gq, gk))
    want = [R.norm_rotary(q, wq, *h, False, EPS, gq), R.norm_rotary(k, wk, *h, False, EPS, gk)]
    bounds = [want[0]["grad"][1], want[1]["grad"][1], want[0]["grad_weight"][1], want[1]["grad_weight"][1]]

    def loss(a, b, c, d):
        one = R.norm_rotary(a, c, *h, False, EPS)["out"][0]
        two = R.norm_rotary(b, d, *h, False, EPS)["out"][0]
        return float((one * gq.double()).sum() + (two * gk.double()).sum())

    step = 1e-4
    for i, g in enumerate(got):
        d = torch.randn_like(leaves[i], dtype=torch.float64)
        base = [t.detach().double() for t in leaves]
        plus, minus = list(base), list(base)
        plus[i], minus[i] = base[i] + step * d, base[i] - step * d
        num = (loss(*plus) - loss(*minus)) / (2 * step)
        limit = float((bounds[i] * d.abs()).sum()) + 1e-6 * float((g.double() * d).abs().sum())
        assert abs(float((g.double() * d).sum()) - num) <= limit
    x = q.clone().requires_grad_()
    gx, = torch.autograd.grad(msda.rotary(x, *h), x, gq)
    assert torch.equal(gx, msda.rotary_backward(gq, *h))


def test_turning_back_is_the_identity(msda):
    x, = make(8, "f32", 2, 100, (4,), 64)
    h = how("far", 2, 100, (16, 16))
    back = msda.rotary_backward(msda.rotary_forward(x, *h), *h)
    # two rotations, each off by its bound times the pair's size (the turned pair is at most sqrt(2) larger)
    bound = 2.5 * (R.TURN + 2.0 ** -24) * R.pair_size(x.double(), 32, False)
    assert ((back - x).abs() <= bound).all()


def test_graph_replay_and_side_stream(msda):
    B, S, M, N, D = 2, 500, 8, 2, 64
    q, k, gq, gk = make(9, "bf16", B, S, (M, N, M, N), D)
    wq, wk = torch.ones((2, D), device=DEV, dtype=q.dtype)
    h = how("float", B, S, (16, 16))

    def both():
        return (*msda.norm_rotary_forward(q, k, wq, wk, *h), *msda.norm_rotary_backward(q, k, wq, wk, *h, gq, gk))

    here = both()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = both()
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(here, side))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = both()
    for t, f in zip((q, k, gq, gk), make(10, "bf16", B, S, (M, N, M, N), D)):
        t.copy_(f)
    g.replay()
    eager = both()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, cap))


def test_empty_tensors(msda):
    h = how("float", 2, 0, (8, 8))
    q, k, gq, gk = make(11, "bf16", 2, 0, (4, 2, 4, 2), 32)
    w = torch.ones(32, device=DEV, dtype=q.dtype)
    oq, ok = msda.norm_rotary_forward(q, k, w, w, *h)
    assert oq.shape == q.shape and ok.shape == k.shape
    got = msda.norm_rotary_backward(q, k, w, w, *h, gq, gk)
    assert not got[2].any() and not got[3].any()
    q, k = make(11, "bf16", 2, 5, (4, 0), 32)
    h = how("float", 2, 5, (8, 8))
    oq, ok = msda.norm_rotary_forward(q, k, w, w, *h)
    R.check(oq, R.norm_rotary(q, w, *h, False, EPS)["out"], "out")
    assert ok.shape == k.shape


def test_offsets_past_32_bits(msda):
    B, S, M, D = 2, 10, 2, 32
    far = 2 ** 31 + 64
    x, = make(12, "bf16", B, S, (M,), D)
    store = torch.empty(far + S * M * D, dtype=x.dtype, device=DEV)
    y = store.as_strided((B, S, M, D), (far, M * D, D, 1))
    y.copy_(x)
    h = how("float", B, S, (8, 8))
    assert torch.equal(msda.rotary_forward(y, *h), msda.rotary_forward(x, *h))
    del store, y
    torch.cuda.empty_cache()


def test_refusals(msda):
    x, = make(13, "bf16", 1, 4, (2,), 32)
    pos, freq, sections = how("float", 1, 4, (8, 8))
    with pytest.raises(ValueError):
        msda.rotary_forward(x[0], pos, freq, sections)
    with pytest.raises(ValueError):
        msda.rotary_forward(x, pos[:, :3], freq, sections)
    with pytest.raises(ValueError):
        msda.rotary_forward(x, pos, freq[:15], sections)
    with pytest.raises(TypeError):
        msda.rotary_forward(x, pos.double(), freq, sections)
    with pytest.raises(ValueError):
        msda.rotary_forward(x.cpu(), pos.cpu(), freq.cpu(), sections)
    with pytest.raises(ValueError):
        msda.rotary(x, pos.clone().requires_grad_(), freq, sections)
    with pytest.raises(msda.MsdaError):
        msda.rotary_forward(x, pos, torch.ones(20, device=DEV), (10, 10))
    w = torch.ones(32, device=DEV, dtype=x.dtype)
    with pytest.raises(TypeError):
        msda.norm_rotary_forward(x, x, w.float(), w, pos, freq, sections)
    with pytest.raises(msda.MsdaError):
        msda.norm_rotary_forward(x, x, w, w, pos, freq, sections, eps=math.nan)
