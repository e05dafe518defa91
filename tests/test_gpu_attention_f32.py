"""binary32 attention at the sizes where it runs on the tensor cores in pieces:
against the definition in 64 bits, and what the pieces cannot hold."""
import math

import pytest

import dense_reference as R
from test_gpu_attention import DEV, both, make, masks, msda  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SIZES = [
    # B, Q, S, M, N, D
    (2, 321, 515, 8, 2, 48), (1, 130, 3001, 8, 8, 64), (4, 129, 257, 16, 16, 7), (1, 3, 20000, 8, 2, 33), (1, 1, 4097, 8, 8, 1),
    (2, 700, 128, 12, 3, 20), (3, 257, 385, 9, 9, 8), (1, 900, 127, 30, 1, 16), (1, 65, 65, 128, 1, 40),
]


@pytest.mark.parametrize("kind", ["", "keys none", "pairs", "keys pairs each causal"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_sizes_and_masks(msda, size, kind):  # noqa: F811
    B, Q, S, M, N, D = size
    q, k, v, do = make(31, "f32", *size)
    kw, ok = masks(kind, 32, B, Q, S, M)
    want = R.attention(q, k, v, do, ok)
    got = both(msda, q, k, v, do, kw)
    for name in want:
        R.check(got[name], want[name], name)


def strided(t):
    """The same values with rows one element longer than their channels (no 16-byte rows)."""
    wide = torch.full(t.shape[:-1] + (t.shape[-1] + 1,), math.nan, device=t.device)
    wide[..., :-1] = t
    return wide[..., :-1]


def test_strides(msda):  # noqa: F811
    q, k, v, do = make(33, "f32", 2, 300, 333, 8, 4, 40)
    want = both(msda, q, k, v, do, {})
    got = both(msda, strided(q), strided(k), strided(v), do, {})
    for name in want:
        assert torch.equal(got[name], want[name]), name


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan, 1e20, -3.4e38])
@pytest.mark.parametrize("where", ["query", "key", "value"])
def test_values_that_no_pieces_hold(msda, where, value):  # noqa: F811
    """One value beyond the pieces' range: what other rows give stays, and its own are those of the definition."""
    B, Q, S, M, N, D = 1, 300, 300, 8, 8, 32
    t = dict(zip(("query", "key", "value", "do"), make(34, "f32", B, Q, S, M, N, D)))
    t[where][0, 17, 3, 5] = value
    q, k, v, do = t["query"], t["key"], t["value"], t["do"]
    out, lse = msda.attention_forward(q, k, v)
    s = torch.einsum("bqmd,bsmd->bmqs", q.double(), k.double()) / math.sqrt(D)
    want = torch.einsum("bmqs,bsmd->bqmd", s.softmax(-1), v.double()).float()   # to binary32: its infinities
    got = out.view(B, Q, M, D)
    # a score beyond 3.4e38 is an infinity in binary32, and a row that holds +inf has no value there (inf - inf): such rows
    # (the largest finite values times a channel above 1) are not asked for
    over = s.isfinite() & (s.abs() * math.sqrt(D) > torch.finfo(torch.float32).max)
    fine = want.isfinite() & ~over.any(-1).transpose(1, 2)[..., None]
    # another head's rows, or those that the value does not reach: as without it, 2^-20 of the largest value
    assert torch.allclose(got[fine], want[fine], rtol=2.0 ** -20, atol=2.0 ** -20 * float(v[v.abs() < 1e3].abs().max()))
    if where == "value" and not math.isnan(value) and math.isinf(value):
        assert (got[..., 3, 5] == value).all()           # p > 0 times an infinity
    if math.isnan(value):
        assert got[~want.isfinite()].isnan().all()
    grads = msda.attention_backward(q, k, v, out, lse, do)
    other = [h for h in range(M) if h != 3]
    for x, y in zip(grads, R_grads(q, k, v, do, other, M, D)):
        assert torch.allclose(x[:, :, other].double(), y, rtol=2.0 ** -16, atol=2.0 ** -16)


def R_grads(q, k, v, do, heads, M, D):
    """Gradients of some heads in 64 bits."""
    q, k, v = (x[:, :, heads].double().requires_grad_() for x in (q, k, v))
    s = torch.einsum("bqmd,bsmd->bmqs", q, k) / math.sqrt(D)
    out = torch.einsum("bmqs,bsmd->bqmd", s.softmax(-1), v)
    out.backward(do.view(*do.shape[:2], M, D)[:, :, heads].double())
    return q.grad, k.grad, v.grad


def test_flag_of_one_call_is_not_the_next_ones(msda):  # noqa: F811
    """One workspace for a call with an infinity and the next without, and a replayed graph whose inputs change."""
    q, k, v, _ = make(35, "f32", 2, 300, 300, 8, 8, 32)
    want = msda.attention_forward(q, k, v)[0]
    bad = v.clone()
    bad[0, 0, 0, 0] = math.inf
    x = v.clone()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        msda.attention_forward(q, k, x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = msda.attention_forward(q, k, x)[0]
    for values, same in ((v, True), (bad, False), (v, True)):
        x.copy_(values)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) == same
        if not same:
            assert (out.view(2, 300, 8, 32)[0, :, 0, 0] == math.inf).all()


def test_sums_over_many_keys_are_not_cut_off(msda):  # noqa: F811
    """20000 keys of one value: each product's sum is cut off on the tensor cores, sums over tiles are not."""
    S = 20000
    q, k = torch.zeros(1, 128, 8, 64, device=DEV), torch.randn(1, S, 8, 64, device=DEV)
    v = torch.full((1, S, 8, 64), 1.0 + 2.0 ** -20, device=DEV)
    out, _ = msda.attention_forward(q, k, v)
    # every probability is 1 / S: eight steps a tile cut off at 2^-23 of its sum at most, the tiles' and rows' sums are
    # rounded (157 and about 160 + 4 halves of 2^-23), the quotient twice
    assert float((out - v[0, 0, 0, 0]).abs().max()) <= (8 + 157 / 2 + 164 / 2 + 1) * 2.0 ** -23
