"""Frequencies of rotary positions against 60 decimal digits, host only."""
from decimal import Decimal, getcontext

import pytest

from bit_matmul_lowbit_amd import lowbit

getcontext().prec = 60
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494")


def frequencies(rot, theta, scaling, factor, trained):
    """Radians a position of each pair."""
    base, by = Decimal(theta), Decimal(factor)
    if scaling == "ntk":
        base *= (by.ln() * rot / (rot - 2)).exp()
    f = [(-base.ln() * 2 * i / rot).exp() for i in range(rot // 2)]
    if scaling == "linear":
        return [v / by for v in f]
    if scaling != "yarn":
        return f
    low, high = ((Decimal(trained) / (beta * 2 * PI)).ln() * rot / (2 * base.ln()) for beta in (32, 1))
    low = max(low.to_integral_value("ROUND_FLOOR"), Decimal(0))
    high = min(high.to_integral_value("ROUND_CEILING"), Decimal(rot - 1))
    mix = [min(max((i - low) / max(high - low, Decimal("0.001")), Decimal(0)), Decimal(1)) for i in range(rot // 2)]
    return [v / by * m + v * (1 - m) for v, m in zip(f, mix)]


@pytest.mark.parametrize("rot,theta,scaling,factor,trained", [
    (2, 10000.0, "none", 1.0, 1), (64, 1e6, "none", 1.0, 1), (128, 1e6, "none", 1.0, 1), (1024, 5e5, "none", 1.0, 1),
    (30, 1.5, "none", 1.0, 1), (128, 10000.0, "linear", 4.0, 1), (80, 1e6, "linear", 3.7, 1), (128, 10000.0, "ntk", 8.0, 1),
    (64, 1e6, "ntk", 2.5, 1), (64, 10000.0, "yarn", 16.0, 4096), (128, 1e6, "yarn", 8.0, 32768), (20, 1.5, "yarn", 3.0, 100)])
def test_turns_to_the_last_bits(rot, theta, scaling, factor, trained):
    """In units of 2^-64 relative: a power's exponent 1, times |ln f|; the power 2; up to five
    products and sums 1 each (two pi's own rounding among them); then half a whole number.  f is at most
    1 and f |ln f| at most 0.37, so f / (2 pi) * 2^64 is off by less than (0.37 + 2 + 5) / (2 pi) + 0.5 < 2."""
    turns, _ = lowbit.lowbit_rope_turns(rot, theta, scaling, factor, trained, device="cpu")
    for t, f in zip(turns.tolist(), frequencies(rot, theta, scaling, factor, trained)):
        assert abs(Decimal(t % 2 ** 64) - f / (2 * PI) * 2 ** 64) < 2


def test_angles_of_far_positions():
    turns, _ = lowbit.lowbit_rope_turns(128, 1e6, device="cpu")
    f = frequencies(128, 1e6, "none", 1.0, 1)
    for position in (262143, 10 ** 9, 2 ** 31 - 1):
        for t, v in zip(turns.tolist(), f):
            off = (position * t - v * position / (2 * PI) * 2 ** 64) % 2 ** 64 / 2 ** 64  # of a turn
            assert min(off, 1 - off) * 2 * PI < Decimal(position) * Decimal(2) ** -63 * 2 * PI
