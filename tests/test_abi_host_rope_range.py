"""Rotary frequencies at the end of their range (no GPU needed): exact up to 2^40 radians a position, refused
past it."""

import random
from fractions import Fraction

import pytest

from test_abi_host_ragged import PI, lib  # noqa: F401


def test_turns_are_exact_up_to_the_largest_frequency(lib):
    """Within one unit of 2^-64 of the doubles' exact product with 1 / 2 pi, modulo 1 (pi to 62 digits: 2^40 / pi
    is off by 2^-160 of a turn there)."""
    rng = random.Random(1)
    freq = [2.0 ** 40, -2.0 ** 40, 2.0 ** 40 - 2.0 ** -13, 2.0 ** 39 + 0.5, 1e12, 1e9 + 1 / 3]
    freq += [rng.choice([1, -1]) * 2.0 ** rng.uniform(-70, 40) for _ in range(3000)]
    for f, t in zip(freq, lib.duo_rope_turns(freq)):
        exact = Fraction(f) / (2 * PI) * 2 ** 64
        off = (t - exact) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= 1, f


@pytest.mark.parametrize("f", [2.0 ** 40 + 2.0 ** -12, -2.0 ** 41, 2.0 ** 50, 2.0 ** 56, 1e30, -1e300, float("-inf")])
def test_larger_frequencies_are_refused(lib, f):
    with pytest.raises(lib.DuoError, match="DUO_ERR_INVALID_ARG.*frequency 2"):
        lib.duo_rope_turns([0.0, 1.0, f])


def test_rope_objects_refuse_them_too(lib):
    from streaming_kv_cache_duo_gb300 import DuoRope
    with pytest.raises(lib.DuoError, match="frequency 7"):
        DuoRope(64, rotary_dim=16, inv_freq=[1.0] * 7 + [1e20], device="cpu")
