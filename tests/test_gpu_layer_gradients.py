"""Gradients through norm, rotation and attention together, against autograd of the formulas in 64 bits."""
import math

import pytest

from test_gpu_attention import DEV, DT, masks, msda  # noqa: F401
import dense_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def plain(q, k, v, wq, wk, pos, freq, sections, interleaved, allowed):
    N, G = k.shape[2], q.shape[2] // k.shape[2]

    def turned(x, w):
        z = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
        return R.turn(z, pos, freq, sections, interleaved)

    q, k = turned(q, wq), turned(k, wk)
    s = torch.einsum("bqmd,bsmd->bmqs", q, k.repeat_interleave(G, 2)) / math.sqrt(q.shape[3])
    if allowed is not None:
        s = s.masked_fill(~allowed, -math.inf)
    return torch.einsum("bmqs,bsmd->bqmd", s.softmax(-1), v.repeat_interleave(G, 2)).flatten(2)


# Each of the three operators sums at most 256 values (2^-23 a step at most: 2^-15), gradients pass five such steps with a factor
# of at most 6 from scores (|s| <= sqrt(32) |wq wk|): 2^-10.  In 16 bits queries, keys, P, dS and every result are rounded, 2^-9 in
# the root mean square in bf16 (2^-12 in f16), a rounded query or key moving a score by that times its size (about 1 here, at most 6): eight
# such roundings add up to 2^-9 * sqrt(8) * 6 = 2^-5 (2^-8) of a gradient's norm.
LIMIT = {"f32": 2.0 ** -10, "f16": 2.0 ** -8, "bf16": 2.0 ** -5}


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind", ["", "keys", "pairs"])
def test_gradients_of_a_layer(msda, kind, interleaved, dtype):  # noqa: F811
    B, Q, M, N, D = 2, 150, 4, 2, 32
    g = torch.Generator(device=DEV).manual_seed(91)
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV).to(DT[dtype])   # noqa: E731
    leaves = [rnd(B, Q, M, D), rnd(B, Q, N, D), rnd(B, Q, N, D), (1 + 0.1 * rnd(D)), (1 + 0.1 * rnd(D))]
    leaves = [t.to(DT[dtype]).requires_grad_() for t in leaves]
    do = rnd(B, Q, M * D)
    pos = torch.rand((B, Q, 2), generator=g, device=DEV) * 50
    freq = (100.0 ** (-torch.arange(8, device=DEV) / 8.0)).repeat(2)
    kw, ok = masks(kind, 92, B, Q, Q, M)
    if "mask" in kw:
        kw["mask"][Q // 2, 0] = True    # no row without keys: their softmax has no value in the plain form
        ok = kw["mask"][None, None]
    q, k = msda.norm_rotary(leaves[0], leaves[1], leaves[3], leaves[4], pos, freq, (8, 8), interleaved=interleaved)
    out = msda.attention(q, k, leaves[2], **kw)
    got = torch.autograd.grad(out, leaves, do)
    exact = [t.detach().double().requires_grad_() for t in leaves]
    ref = plain(*exact, pos, freq, (8, 8), interleaved, ok)
    want = torch.autograd.grad(ref, exact, do.double())
    out, ref = out.detach(), ref.detach()
    for name, a, b in zip(("out", "query", "key", "value", "query weight", "key weight"), (out, *got), (ref, *want)):
        assert float((a.double() - b).norm() / b.norm()) <= LIMIT[dtype], name
