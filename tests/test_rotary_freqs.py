"""The frequencies of rotary positions: 64-bit fractions of a turn, rounded once.  CPU
only."""
import math
from fractions import Fraction

import pytest

import fp8_w8a8_rollout_gb300 as fp8rl

# pi to 100 decimals
PI = Fraction(int("31415926535897932384626433832795028841971693993751058209749445923078164062862089986280348253421170680"), 10 ** 100)


def exact(f):
    """f / (2 pi) modulo 1 in units of 2^-64, to the nearest (pi above holds for |f| up to 2^200)."""
    return round(Fraction(f) / (2 * PI) * 2 ** 64) % 2 ** 64


def words(freqs):
    return [w % 2 ** 64 for w in freqs.data[0].tolist()]


@pytest.mark.parametrize("theta", [10000.0, 500000.0, 1e6])
@pytest.mark.parametrize("dim", [8, 64, 128])
def test_powers_of_theta(theta, dim):
    pairs = dim // 2
    assert words(fp8rl.rotary_freqs(dim, theta, device="cpu")) == [exact(theta ** (-i / pairs)) for i in range(pairs)]


def test_given_frequencies():
    inv = [1.0, -1.0, 2.5, 7.5, 100.0, -1234.5678, 0.0, -0.0, 1e-9, 2.0 ** -70, 5e-324, 1e15, 2.0 ** 64, -1e50, math.pi, 2 * math.pi, 0.1]
    inv.append(3.0)
    assert words(fp8rl.rotary_freqs(2 * len(inv), inv_freq=inv, device="cpu")) == [exact(f) for f in inv]


def test_the_angle_at_the_last_position():
    # 2^-65 of a turn a position: 2^-34 at 2^31
    for f in (1.0, 2.5, 0.7498942093324559, -3.75):
        word = words(fp8rl.rotary_freqs(2, inv_freq=[f], device="cpu"))[0]
        for p in (2 ** 31 - 1, -2 ** 31):
            off = (p * Fraction(f) / (2 * PI) - Fraction(p * word, 2 ** 64)) % 1
            assert min(off, 1 - off) <= Fraction(1, 2 ** 34)
