"""The dense operators' C ABI on the host, without a GPU: sizes of workspaces
and refusals.  No call here reaches a launch: each fails validation first."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    from scale_deformable_attention_gb300 import _lib, build

    build.build()
    return _lib.lib()


def attention_problem(B=2, Q=10, S=12, M=4, N=2, D=32, q=None, k=None, v=None, km=None, ms=(0, 0, 0)):
    from scale_deformable_attention_gb300._lib import AttentionProblem

    dense = lambda rows, heads: (rows * heads * D, heads * D, D)     # noqa: E731
    q, k, v = q or dense(Q, M), k or dense(S, N), v or dense(S, N)
    return AttentionProblem(B, Q, S, M, N, D, *q, *k, *v, S if km is None else km, *ms)


def forward(lib, p, dt=2, flags=0, scale=1.0, ptrs=None, ws=None, n=0):
    a = {"query": FAKE, "key": FAKE, "value": FAKE, "key_mask": None, "mask": None, "out": FAKE, "lse": FAKE}
    a.update(ptrs or {})
    return lib.msda_attention_forward(dt, flags, p, scale, *a.values(), ws, n, None)


def backward(lib, p, dt=2, flags=0, scale=1.0, ptrs=None, ws=None, n=0):
    a = {"query": FAKE, "key": FAKE, "value": FAKE, "key_mask": None, "mask": None, "out": FAKE, "lse": FAKE,
         "grad_out": FAKE, "grad_query": FAKE, "grad_key": FAKE, "grad_value": FAKE}
    a.update(ptrs or {})
    return lib.msda_attention_backward(dt, flags, p, scale, *a.values(), ws, n, None)


def msg(lib):
    return lib.msda_last_error().decode()


@pytest.mark.parametrize("call", [forward, backward])
@pytest.mark.parametrize("kw,status,text", [
    (dict(B=-1), 1, "negative"), (dict(M=0), 1, "at least 1"), (dict(N=0), 1, "at least 1"), (dict(D=0), 1, "at least 1"),
    (dict(M=4, N=3), 1, "divide"), (dict(D=129), 2, "D=129"), (dict(Q=1 << 31), 2, "too large"),
    (dict(S=1 << 31), 2, "too large"), (dict(B=1 << 30, Q=1 << 30, M=60000, N=1), 1, "overflow"),
    (dict(B=1 << 20, Q=1 << 20, M=1, N=1), 2, "blocks"), (dict(q=(-1, 1, 1)), 1, "negative stride"),
    (dict(km=-1), 1, "negative stride"), (dict(ms=(0, -1, 0)), 1, "negative stride"),
])
def test_attention_rejects_sizes(lib, call, kw, status, text):
    assert call(lib, attention_problem(**kw)) == status
    assert text in msg(lib)


@pytest.mark.parametrize("call", [forward, backward])
def test_attention_rejects_arguments(lib, call):
    p = attention_problem()
    assert call(lib, p, dt=5) == 1 and "dtype" in msg(lib)
    assert call(lib, p, flags=8) == 1 and "flags" in msg(lib)
    assert call(lib, None) == 1 and "problem" in msg(lib)
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(lib, p, scale=scale) == 1 and "scale" in msg(lib)
    assert call(lib, p, flags=2) == 1 and "key_mask" in msg(lib)
    assert call(lib, p, flags=4) == 1 and "mask" in msg(lib)
    assert call(lib, p, ptrs={"mask": FAKE}) == 1 and "flag" in msg(lib)
    assert call(lib, p, ptrs={"key_mask": FAKE}) == 1 and "flag" in msg(lib)


@pytest.mark.parametrize("name", ["query", "key", "value", "out", "lse"])
def test_attention_rejects_pointers(lib, name):
    p = attention_problem()
    for call in (forward, backward):
        assert call(lib, p, ptrs={name: None}) == 1 and name in msg(lib)
        assert call(lib, p, ptrs={name: FAKE + 1}) == 3 and name in msg(lib)


def test_attention_workspace(lib):
    p = attention_problem()
    for dt in (0, 1, 2):
        need = lib.msda_attention_backward_workspace_size(dt, 0, p)
        assert need >= 2 * 2 * 4 * 10 * 4
        assert backward(lib, p, dt=dt) == 4 and "workspace" in msg(lib)
        assert backward(lib, p, dt=dt, ws=FAKE, n=need - 1) == 4
        assert backward(lib, p, dt=dt, ws=FAKE + 16, n=need) == 4
    assert lib.msda_attention_forward_workspace_size(2, 0, p) == 0       # few keys: no split, no mask
    long = attention_problem(B=1, Q=1, S=20000, M=8, N=2)
    assert lib.msda_attention_forward_workspace_size(2, 0, long) >= 8 * 33 * 4
    assert forward(lib, long) == 4 and "workspace" in msg(lib)
    m = attention_problem(ms=(0, 0, 12))
    assert lib.msda_attention_forward_workspace_size(2, 4, m) >= 12 + 10 * 16 + 12 * 16
    assert lib.msda_attention_forward_workspace_size(2, 0, attention_problem(D=200)) == 0


def test_attention_of_nothing_is_ok(lib):
    null = dict.fromkeys(("query", "key", "value", "out", "lse"))
    assert forward(lib, attention_problem(B=0), ptrs=null) == 0
    assert forward(lib, attention_problem(Q=0), ptrs=null) == 0
    grads = dict.fromkeys(("query", "key", "value", "out", "lse", "grad_out", "grad_query", "grad_key", "grad_value"))
    assert backward(lib, attention_problem(B=0), ptrs=grads) == 0


def rotary_problem(B=2, S=10, M=4, N=2, D=32, axes=2, sections=(8, 8, 0, 0), q=None, k=None, pt=0, ps=0):
    from scale_deformable_attention_gb300._lib import RotaryProblem

    q, k = q or (S * M * D, M * D, D), k or (S * N * D, N * D, D)
    return RotaryProblem(B, S, M, N, D, axes, *sections, *q, *k, pt, ps)


def rotary(lib, p, dt=2, flags=0, eps=1e-6, ptrs=None):
    a = dict(positions=FAKE, frequencies=FAKE, query=FAKE, key=FAKE, query_weight=FAKE, key_weight=FAKE, query_out=FAKE,
             key_out=FAKE)
    a.update(ptrs or {})
    return lib.msda_norm_rotary_forward(dt, flags, p, eps, *a.values(), None)


def rotary_back(lib, p, dt=2, flags=0, eps=1e-6, ptrs=None, ws=None, n=0):
    a = dict(positions=FAKE, frequencies=FAKE, query=FAKE, key=FAKE, query_weight=FAKE, key_weight=FAKE,
             grad_query_out=FAKE, grad_key_out=FAKE, grad_query=FAKE, grad_key=FAKE, grad_query_weight=FAKE,
             grad_key_weight=FAKE)
    a.update(ptrs or {})
    return lib.msda_norm_rotary_backward(dt, flags, p, eps, *a.values(), ws, n, None)


@pytest.mark.parametrize("call", [rotary, rotary_back])
@pytest.mark.parametrize("kw,status,text", [
    (dict(B=-1), 1, "negative"), (dict(D=257), 2, "D=257"), (dict(axes=0), 2, "axes"), (dict(axes=5), 2, "axes"),
    (dict(sections=(-1, 8, 0, 0)), 1, "section"), (dict(sections=(9, 8, 0, 0)), 1, "pairs"), (dict(pt=3), 1, "position"),
    (dict(q=(1, -1, 1)), 1, "stride"), (dict(ps=-1), 1, "stride"), (dict(S=1 << 31), 2, "too large"),
    (dict(B=1 << 62), 1, "overflow"),
])
def test_rotary_rejects_sizes(lib, call, kw, status, text):
    assert call(lib, rotary_problem(**kw)) == status
    assert text in msg(lib)


def test_rotary_rejects_arguments(lib):
    p = rotary_problem()
    for call in (rotary, rotary_back):
        assert call(lib, p, dt=3) == 1 and "dtype" in msg(lib)
        assert call(lib, p, flags=4) == 1 and "flags" in msg(lib)
        assert call(lib, None) == 1 and "problem" in msg(lib)
        for eps in (-1.0, float("nan")):
            assert call(lib, p, eps=eps) == 1 and "eps" in msg(lib)
        for name in ("positions", "frequencies", "query", "key"):
            assert call(lib, p, ptrs={name: None}) == 1 and name in msg(lib)
            assert call(lib, p, ptrs={name: FAKE + 1}) == 3 and name in msg(lib)
        assert call(lib, p, ptrs={"key_weight": None}) == 1 and "key_weight" in msg(lib)   # one weight alone
    assert rotary_back(lib, p, flags=2) == 1 and "INVERSE" in msg(lib)
    need = lib.msda_norm_rotary_backward_workspace_size(p)
    assert need > 0
    assert rotary_back(lib, p) == 4 and rotary_back(lib, p, ws=FAKE, n=need - 1) == 4


def test_rotary_of_nothing_is_ok(lib):
    null = dict.fromkeys(("positions", "frequencies", "query", "key", "query_weight", "key_weight", "query_out", "key_out"))
    assert rotary(lib, rotary_problem(B=0), ptrs=null) == 0
    assert rotary(lib, rotary_problem(M=0, N=0), ptrs=null) == 0
    assert lib.msda_norm_rotary_backward_workspace_size(rotary_problem(S=0)) == 0


def test_kernel_names(lib):
    from scale_deformable_attention_gb300 import _lib

    for i, name in _lib.KERNEL_NAMES.items():
        assert lib.msda_kernel_name(i).decode() == name


def test_binding_refuses_cpu_tensors():
    import scale_deformable_attention_gb300 as msda

    q = torch.zeros(1, 2, 1, 8)
    with pytest.raises(ValueError):
        msda.attention_forward(q, q, q)
    with pytest.raises(ValueError):
        msda.rotary_forward(q, torch.zeros(1, 2, 1), torch.ones(4), (4,))
    with pytest.raises(TypeError):
        msda.norm_rotary_forward(q, None, None, None, torch.zeros(1, 2, 1), torch.ones(4), (4,))
    assert ctypes.sizeof(msda._lib.AttentionProblem) == 19 * 8 and ctypes.sizeof(msda._lib.RotaryProblem) == 18 * 8
