"""The factor of the rotated pairs under "yarn": 0.1 ln(s) + 1 for contexts stretched by s > 1, and 1 where
nothing is stretched."""

import math

import pytest


@pytest.mark.parametrize("s,factor", [(0.25, 1.0), (0.5, 1.0), (1.0, 1.0), (1, 1.0), (math.e, 1.1), (40.0, 0.1 * math.log(40.0) + 1)])
def test_factor_of_rotated_pairs(s, factor):
    from streaming_kv_cache_duo_gb300 import rope_frequencies
    freq, got = rope_frequencies(64, 10000.0, dict(kind="yarn", factor=s, original=4096))
    assert math.isclose(got, factor, rel_tol=1e-15)
    assert freq[0] == 1.0 and math.isclose(freq[-1], 10000.0 ** (-31 / 32) / s)
