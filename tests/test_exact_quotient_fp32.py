"""The division-free quotient on fp32 values (the experts' h is quantized from fp32, not from bf16).

The argument of test_exact_quotient_method.py does not use the eight bits of a bf16 significand: the residual
of a faithful quotient is exact for any binary32 x while nothing underflows. Checked here in the same exact
arithmetic on random binary32 values of a block, on values a few ulps around every e4m3 rounding boundary,
and at the ends of the scales the form is used for; and the codes, which have to be those of the IEEE
quotient also where the quotient itself may differ (below 2**-20: both give code 0)."""

import numpy as np
import pytest

from oracle import fp8_oracle as O
from test_exact_quotient_method import check_scale, kernel_quotient


def codes_agree(s, xs):
    s = np.float32(s)
    with np.errstate(under="ignore"):
        ref = O.encode((xs / s).astype(np.float32))
    got = O.encode(np.array([kernel_quotient(float(x), float(s)) for x in xs], np.float32))
    same = (ref == got) | ((ref & 0x7F) == 0) & ((got & 0x7F) == 0)  # -0 and +0 are the same value
    assert same.all(), f"s={s!r}: x={xs[~same][:3].tolist()}"


def boundaries():
    """Midpoints between neighbouring e4m3 magnitudes: where a code changes."""
    v = O.decode(np.arange(0x7F, dtype=np.uint8)).astype(np.float64)  # 0 .. 448
    return (v[:-1] + v[1:]) / 2


def block_scale(amax):
    return float(np.float32(amax) / np.float32(448.0))


@pytest.mark.parametrize("seed", range(6))
def test_random_blocks(seed):
    g = np.random.default_rng(seed)
    amax = np.float32(np.exp2(g.uniform(-60, 60)))
    xs = (g.uniform(-1, 1, 3000) * amax).astype(np.float32)
    xs = np.concatenate([xs, (xs[:1000] * np.exp2(g.integers(-30, 0, 1000))).astype(np.float32), [amax, -amax]])
    xs = xs[xs != 0]
    assert check_scale(block_scale(amax), xs) > 2000
    codes_agree(block_scale(amax), xs)


@pytest.mark.parametrize("amax", [448.0, 3.375, 7.0 * 2.0 ** -9, float(np.float32(0.1)), float(np.float32(np.pi)) * 2.0 ** 40])
def test_around_every_boundary(amax):
    s = block_scale(amax)
    xs = []
    for m in boundaries():
        x = np.float32(m * s)
        xs.append(x)
        for up in (np.float32(np.inf), np.float32(0)):
            y = x
            for _ in range(3):
                y = np.nextafter(y, up)
                xs.append(y)
    xs = np.array(xs, np.float32)
    xs = np.concatenate([xs, -xs])
    assert check_scale(s, xs) > 1000
    codes_agree(s, xs)


@pytest.mark.parametrize("s", [2.0 ** -80, float(np.nextafter(np.float32(2.0 ** -80), np.float32(1))), 2.0 ** 100,
                               float(np.nextafter(np.float32(2.0 ** 100), np.float32(0)))])
def test_ends_of_the_range(s):
    g = np.random.default_rng(11)
    q = np.concatenate([g.uniform(2.0 ** -12, 448, 1500), np.exp2(g.uniform(-20, 8.8, 500))])
    xs = (q * s).astype(np.float32)
    assert check_scale(s, xs) > 1900
    codes_agree(s, np.concatenate([xs, (np.exp2(g.uniform(-60, -20, 300)) * s).astype(np.float32)[:300]]))
