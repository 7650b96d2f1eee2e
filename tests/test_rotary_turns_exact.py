"""Frequencies as fractions of a turn, against whole-number arithmetic with 60
digits of pi (CPU only)."""

from fractions import Fraction

import pytest
import torch

import pagedattention_decode_attention_gb300 as pa

TURN = 2 * Fraction(3141592653589793238462643383279502884197169399375105820974944, 10 ** 60)

RANGES = {
    "short": dict(base=10000.0), "long": dict(base=500000.0), "far": dict(base=1e6),
    "linear": dict(base=10000.0, scaling="linear", factor=3.5),
    "base": dict(base=10000.0, scaling="base", factor=8.0),
    "bands": dict(base=500000.0, scaling="bands", factor=8.0, original_context=8192, low=1.0, high=4.0),
}


def exact(w):
    """The frequency's fraction of a turn, times 2^64 (a rational)."""
    return Fraction(w) / TURN % 1 * 2 ** 64


@pytest.mark.parametrize("name", sorted(RANGES))
@pytest.mark.parametrize("rotary_dim", [16, 112, 128])
def test_a_frequency_is_rounded_once(name, rotary_dim):
    w = pa.rotary_frequencies(rotary_dim, **RANGES[name])
    for sign in (1.0, -1.0):
        for x, t in zip((sign * w).tolist(), pa.rotary_turns(sign * w).tolist()):
            off = (t - exact(x) + 2 ** 63) % 2 ** 64 - 2 ** 63
            # half a unit, and the quotient's own error: under 2^-102 of it, 2^-38 units
            assert abs(off) <= Fraction(1, 2) + Fraction(1, 2 ** 30)


@pytest.mark.parametrize("x", [0.0, 5e-324, 1e-30, 2.0 ** -60, 1e-9, 3.141592653589793, 6.283185307179586, 12345.678,
                               -98765.4321, 2.0 ** 40 + 0.3])
def test_any_frequency(x):
    t = int(pa.rotary_turns(torch.tensor([x], dtype=torch.float64))[0])
    off = (t - exact(x) + 2 ** 63) % 2 ** 64 - 2 ** 63
    # (2^64 * 2^-102 of the quotient)
    assert abs(off) <= Fraction(1, 2) + Fraction(abs(x)) * Fraction(1, 2 ** 38)


@pytest.mark.parametrize("position", [1, -1, 65536, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31])
def test_angles_at_any_position(position):
    """position * turns is within 2^-33 of a turn of the exact angle."""
    w = pa.rotary_frequencies(128, 500000.0)
    for x, t in zip(w.tolist(), pa.rotary_turns(w).tolist()):
        got = Fraction(position * t % 2 ** 64, 2 ** 64)
        off = (got - Fraction(x) / TURN * position + Fraction(1, 2)) % 1 - Fraction(1, 2)
        assert abs(off) <= Fraction(1, 2 ** 33)
