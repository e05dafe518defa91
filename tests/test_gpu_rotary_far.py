"""Rotary positions far out, against angles that integer arithmetic reduces."""
import math

import pytest

from test_gpu_rotary import DEV, msda  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def two_pi(bits):
    """2 pi times 2^bits as an integer, by Machin's 16 atan(1/5) - 4 atan(1/239)."""
    one = 1 << (bits + 16)

    def atan_inverse(n):
        total, term, k, sign = 0, one // n, 1, 1
        while term:
            total += sign * (term // k)
            term, k, sign = term // (n * n), k + 2, -sign
        return total

    return 2 * (16 * atan_inverse(5) - 4 * atan_inverse(239)) >> 16


BITS = 200
TWO_PI = two_pi(BITS)


def angle(position, frequency):
    """position * frequency modulo 2 pi: both are whole numbers times a power of two, so the product is exact."""
    fn, fd = frequency.as_integer_ratio()
    pn, pd = position.as_integer_ratio()
    return ((pn * fn << BITS) // (pd * fd)) % TWO_PI / (1 << BITS)


def test_two_pi():
    assert TWO_PI / (1 << BITS) == 2 * math.pi


FREQUENCIES = [1.0, 0.7310586, 0.333333343, 1e-3, 1.1920929e-07, 3.1415927, 2.5e-5, 0.9999999]
SMALL = [2.0 ** -13 * 1.2345678, 2.0 ** -14, 1e-5, 1.7e-7, 2.0 ** -13, 3e-5, 2.0 ** -20, 1.2e-4]   # times 2^63: below 2^51
POSITIONS = {
    "int32": ([2 ** 31 - 1, -2 ** 31, 2 ** 29 + 12345, 1234567891, 16777217, -16777219], torch.int32, FREQUENCIES),
    "int64": ([2 ** 33 + 1, -(2 ** 37) - 3, 2 ** 40 + 987654321, 2 ** 45 - 1, 2 ** 49 + 12345677, -(2 ** 49) + 5,
               2 ** 48 + 2 ** 20 + 1], torch.int64, FREQUENCIES),
    "no binary64": ([2 ** 62 + 1025, -(2 ** 60) - 1, 2 ** 63 - 1, -(2 ** 63) + 1, 2 ** 53 + 1], torch.int64, SMALL),
    "float32": ([2.0 ** 23 + 1, 1.5e9, -7.7e11, 3.3e14, 123456.789], torch.float32, FREQUENCIES),
}


@pytest.mark.parametrize("kind", list(POSITIONS))
@pytest.mark.parametrize("D,interleaved", [(32, False), (32, True), (20, False)])
def test_far_positions(msda, kind, D, interleaved):  # noqa: F811
    """Angles up to 2^51; (1, 0) turned is cos and sin themselves.  The reduced angle is below 8 and rounded to binary32 once
    (2^-22; two roundings below 4 and the rest of 2 pi, 2^-27, for angles up to 2^23), sincosf is off by two steps (2^-23)."""
    P = D // 4
    values, dtype, f = POSITIONS[kind]
    pos, f, S = torch.tensor(values, dtype=dtype), torch.tensor(f[:P], dtype=torch.float32), len(values)
    u, v = (slice(0, 2 * P, 2), slice(1, 2 * P, 2)) if interleaved else (slice(0, P), slice(P, 2 * P))
    x = torch.zeros(1, S, 1, D, device=DEV)
    x[..., u] = 1
    out = msda.rotary_forward(x, pos.view(1, S, 1).to(DEV), f.to(DEV), (P,), interleaved=interleaved).cpu()[0, :, 0]
    for i in range(S):
        for j in range(P):
            t = angle(pos[i].item(), f[j].item())
            for got, want in ((out[i, u][j], math.cos(t)), (out[i, v][j], math.sin(t))):
                assert abs(float(got) - want) <= 2.0 ** -22 + 2.0 ** -23 + 2.0 ** -27, (pos[i].item(), f[j].item())
