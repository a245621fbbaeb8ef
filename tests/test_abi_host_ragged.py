"""Rotary positions and packed steps on the host (no GPU needed): frequencies, their fixed-point form, and
what the entry points refuse before they touch a device."""

import math
from fractions import Fraction

import pytest

PI = Fraction(314159265358979323846264338327950288419716939937510582097494459, 10 ** 62)


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    from streaming_kv_cache_duo_gb300 import _lib
    return _lib


def test_turns_are_the_frequencies_as_fractions_of_a_turn(lib):
    """Within one unit of 2^-64 of the exact value (the doubles' exact product with 1 / 2 pi, modulo 1), also
    above a turn, below zero and at the borders."""
    freq = [0.0, 1.0, 1e-30, 0.7, 2 * math.pi, 6.3, 1234.5678, -0.25, -1e-12] + \
        [10000.0 ** (-2 * i / 128) for i in range(64)] + [1e6 ** (-2 * i / 96) for i in range(48)]
    for f, t in zip(freq, lib.duo_rope_turns(freq)):
        exact = Fraction(f) / (2 * PI) * 2 ** 64
        off = (t - exact) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= 1, f


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_turns_refuse_what_is_not_finite(lib, bad):
    with pytest.raises(lib.DuoError, match="DUO_ERR_INVALID_ARG"):
        lib.duo_rope_turns([1.0, bad])


def test_frequencies():
    from streaming_kv_cache_duo_gb300 import rope_frequencies
    plain, one = rope_frequencies(64, 10000.0)
    assert one == 1.0 and plain[0] == 1.0 and len(plain) == 32
    assert all(math.isclose(f, 10000.0 ** (-i / 32)) for i, f in enumerate(plain))
    linear, one = rope_frequencies(64, 10000.0, dict(kind="linear", factor=4))
    assert one == 1.0 and all(math.isclose(a, b / 4) for a, b in zip(linear, plain))
    ntk, one = rope_frequencies(64, 10000.0, dict(kind="ntk", factor=8.0))
    # the fastest pair keeps its frequency, the slowest has it divided by the factor
    assert one == 1.0 and ntk[0] == 1.0 and math.isclose(ntk[-1], plain[-1] / 8)
    wl, one = rope_frequencies(64, 10000.0, dict(kind="wavelength", factor=8.0, low=1.0, high=4.0, original=8192))
    for f, g in zip(plain, wl):
        turns = 8192 * f / (2 * math.pi)
        if turns >= 4:
            assert g == f
        elif turns <= 1:
            assert math.isclose(g, f / 8)
        else:
            w = (turns - 1) / 3
            assert math.isclose(g, w * f + (1 - w) * f / 8)
    yarn, factor = rope_frequencies(64, 10000.0, dict(kind="yarn", factor=16.0, original=4096))
    assert math.isclose(factor, 0.1 * math.log(16) + 1)
    at = lambda n: 64 * math.log(4096 / (n * 2 * math.pi)) / (2 * math.log(10000.0))
    lo, hi = math.floor(at(32)), math.ceil(at(1))
    for i, (f, g) in enumerate(zip(plain, yarn)):
        w = min(1, max(0, (i - lo) / (hi - lo)))
        assert math.isclose(g, f * (1 - w) + f / 16 * w)
    assert yarn[0] == 1.0 and math.isclose(yarn[-1], plain[-1] / 16)


@pytest.mark.parametrize("scaling", [dict(kind="other", factor=2), dict(factor=2), dict(kind="linear"),
                                     dict(kind="linear", factor=0), dict(kind="linear", factor="4"),
                                     dict(kind="linear", factor=2, original=5), dict(kind="yarn", factor=2),
                                     dict(kind="wavelength", factor=2, low=4, high=1, original=100)])
def test_frequencies_refuse(scaling):
    from streaming_kv_cache_duo_gb300 import rope_frequencies
    with pytest.raises(ValueError):
        rope_frequencies(64, 10000.0, scaling)


def test_theta_of_one_or_less_is_refused():
    from streaming_kv_cache_duo_gb300 import rope_frequencies
    with pytest.raises(ValueError):
        rope_frequencies(64, 1.0)


def _rotate(lib, head_dim=64, tokens=4, rotary=64, layout=0, scale=1.0, hq=2, hk=1, stride=128, out_stride=128, null=None,
            off=None):
    from ctypes import byref, c_void_p
    at = {n: 0x10000 * (i + 1) for i, n in enumerate(("turns", "pos", "q", "qo", "k", "ko"))}
    if null:
        at[null] = None
    if off:
        at[off] += 4 if off != "pos" else 2
    rope = lib.duo_rope(at["turns"], rotary, layout, scale)
    p = lambda n: c_void_p(at[n])
    return lib.library().duo_rope_rotate(byref(rope), head_dim, p("pos"), tokens, p("q"), stride, p("qo"), out_stride, hq,
                                         p("k"), 64 if head_dim == 64 else 128, p("ko"), 128, hk, None)


@pytest.mark.parametrize("args,status", [
    (dict(head_dim=80), 2), (dict(tokens=-1), 1), (dict(rotary=72), 1), (dict(rotary=0), 1), (dict(rotary=24), 2),
    (dict(layout=2), 1), (dict(scale=float("nan")), 1), (dict(hq=0), 1), (dict(hk=0), 1), (dict(stride=120), 1),
    (dict(stride=132), 1), (dict(out_stride=64), 1), (dict(null="turns"), 1), (dict(null="pos"), 1), (dict(null="q"), 1),
    (dict(null="qo"), 1), (dict(null="ko"), 1), (dict(off="turns"), 1), (dict(off="pos"), 1), (dict(off="q"), 1),
    (dict(off="ko"), 1), (dict(tokens=0), 0), (dict(tokens=0, rotary=24), 2),
])
def test_rotation_refusals(lib, args, status):
    assert _rotate(lib, **args) == status
    assert (lib.duo_last_error() != "") == (status != 0)


def test_rotation_in_place_with_another_stride_is_refused(lib):
    from ctypes import byref
    rope = lib.duo_rope(0x10000, 64, 0, 1.0)
    call = lambda out_stride: lib.library().duo_rope_rotate(byref(rope), 64, 0x20000, 4, 0x30000, 128, 0x30000, out_stride,
                                                            2, None, 0, None, 0, 0, None)
    assert call(256) == 1 and "in place" in lib.duo_last_error()


def test_packed_entry_points_refuse_a_null_handle(lib):
    import ctypes
    cache, paged, m = lib.duo_kv_cache(), lib.duo_paged(), lib.duo_slot_map()
    ref = ctypes.byref
    L = lib.library()
    assert L.duo_kv_append_ragged(None, ref(cache), ref(paged), ref(m), 1, None, None, 0, None, 0, None, 0, None, 0, None) == 1
    assert L.duo_attn_prefill_ragged(None, ref(cache), ref(paged), ref(m), 1, None, 0, None, 0, None, 0, None, None, 0, None) == 1
    assert L.duo_attn_decode_paged_varlen(None, ref(cache), ref(paged), None, 1, None, None, None, 0, None) == 1
    assert lib.duo_prefill_ragged_workspace_size(None, 100) == 0


def test_null_rope_is_refused(lib):
    assert lib.library().duo_rope_rotate(None, 64, 0x1000, 1, 0x1000, 64, 0x1000, 64, 1, None, 0, None, 0, 0, None) == 1
