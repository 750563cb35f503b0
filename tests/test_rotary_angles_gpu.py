"""Rotary positions at positions far out, where a 64-bit floating point angle
has too few bits: against the angle in rational numbers."""
import math
from fractions import Fraction

import pytest
import torch

import gated_delta_rule_32_gb300 as pkg
from gated_delta_rule_32_gb300 import kda

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_32_gb300 import build
    build.build()
    kda.load()


def pi():
    # 16 atan(1/5) - 4 atan(1/239) in units of 10^-80
    one = 10 ** 90

    def atan(n):
        total, term, i = 0, one // n, 1
        while term:
            total += term // i if i % 4 == 1 else -(term // i)
            term //= n * n
            i += 2
        return total
    return Fraction(16 * atan(5) - 4 * atan(239), one)


PI = pi()


def angle(pos, f):
    """pos * f modulo 2 pi, in (-pi, pi], to 2^-53."""
    t = Fraction(f) * pos
    t -= round(t / (2 * PI)) * 2 * PI
    return float(t)


def test_the_reference():
    assert abs(float(PI) - math.pi) == 0 and str(int(PI * 10 ** 20)) == "314159265358979323846"
    for p, f in ((0, 3.0), (7, 0.25), (1000, 1.0)):
        assert math.isclose(math.sin(angle(p, f)), math.sin(p * f), abs_tol=1e-12)


FREQS = {
    "base": [10000.0 ** (-i / 8) for i in range(8)],
    "fast": [100.0, 7.5, 2 * math.pi, 63.1, 1.0, 31.4159, 0.75, 99.99],
    "whole": [0.0, 2 * math.pi, 4 * math.pi, math.pi, 1e6 + 0.1, 12345.678, 1e-9, 5e-324],
    "back": [-100.0, -1.0, -1e-20, -0.001, -7.25, -2 * math.pi, -0.0, -1e6],
}


@pytest.mark.parametrize("name", sorted(FREQS))
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_angles_far_out(name, interleaved, dtype):
    # the fraction of a turn errs by 2^-32 (position times 2^-64 in each of two parts), as an fp32
    # number of half turns by 2^-25 of one: 2^-23.3 of a radian together; sine and cosine by two ulp
    # of 1 at most, 2^-23; amplitude, products and their sum by four roundings of 2^-24.  In all
    # less than 2^-20.5 of the pair's length, beside the output's own rounding
    freqs = FREQS[name]
    pos = [0, 1, 2, 1000, 65537, 1 << 20, 10 ** 6 + 3, 1 << 24, (1 << 30) + 1, (1 << 31) - 1, (1 << 31) - 2,
           1987654321, 1 << 30, 1555555555]
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(len(pos), 3, 32, generator=g, device="cuda").to(dtype)
    f = torch.tensor(freqs, dtype=torch.float64, device="cuda")
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    half = torch.finfo(dtype).eps / 2
    for inverse in (False, True):
        got, _ = pkg.rotary_embed(x, None, p, f, interleaved=interleaved, inverse=inverse, amplitude=1.25)
        got, y = got.double().cpu(), x.double().cpu()
        for t, at in enumerate(pos):
            for i, w in enumerate(freqs):
                a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 8)
                r = angle(at, w) * (-1 if inverse else 1)
                c, s = 1.25 * math.cos(r), 1.25 * math.sin(r)
                want = torch.stack([y[t, :, a] * c - y[t, :, b] * s, y[t, :, a] * s + y[t, :, b] * c])
                size = 1.25 * (y[t, :, a] ** 2 + y[t, :, b] ** 2).sqrt()
                err = (torch.stack([got[t, :, a], got[t, :, b]]) - want).abs()
                tol = half * want.abs() + (1 + half) * 2.0 ** -20.5 * size
                assert (err <= tol).all(), (at, w, (err / tol).max())
        assert torch.equal(got[..., 16:], y[..., 16:])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_frequencies_that_are_no_numbers(dtype):
    # as a position times an infinity or a NaN has no sine: the pair is NaN, at position 0 too,
    # and nothing else is
    x = torch.ones(3, 2, 48, dtype=dtype, device="cuda")
    f = torch.full((16,), 0.5, dtype=torch.float64, device="cuda")
    f[2], f[5], f[11] = math.inf, -math.inf, math.nan
    p = torch.tensor([0, 1, 1 << 30], dtype=torch.int32, device="cuda")
    for interleaved in (False, True):
        y, _ = pkg.rotary_embed(x, None, p, f, interleaved=interleaved)
        bad = {(2 * i + k) if interleaved else (i + 16 * k) for i in (2, 5, 11) for k in (0, 1)}
        want = torch.tensor([c in bad for c in range(48)], device="cuda").expand(3, 2, 48)
        assert torch.equal(y.isnan(), want) and bool(y[~want].isfinite().all())
