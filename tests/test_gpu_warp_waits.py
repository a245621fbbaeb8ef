"""A bounded wait that guards warp-wide instructions has one answer for the whole warp: the self-test
lets the lanes' times end apart, with the barrier completed in between, and records lanes that part
ways (bit 17)."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("limit_us", [400, 20000])
def test_a_warp_waits_with_one_answer(limit_us):
    from streaming_kv_cache_duo_gb300 import _lib
    assert _lib.duo_device_error() == 0
    for _ in range(3):
        _lib.duo_selftest_bounded_wait(limit_us)
        assert _lib.duo_device_error() == 1 << 16
    assert _lib.duo_device_error() == 0
