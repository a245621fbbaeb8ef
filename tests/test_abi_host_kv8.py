"""The 8-bit cache and block table entry points on the host (no GPU needed): what they refuse
before they touch a device."""

import pytest


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    from streaming_kv_cache_duo_gb300 import _lib
    return _lib


def _tables_call(lib, batch=4, planes=2, block_size=128, max_blocks=8, num_blocks=64, max_tokens=32, ws=1 << 20,
                 null=None, off=None):
    """duo_block_tables_update with made-up device addresses (never dereferenced on the host)."""
    from ctypes import byref, c_void_p
    at = {n: 0x10000 * (i + 1) for i, n in enumerate(("table", "free", "count", "lens", "new", "lens_out", "count_out",
                                                      "cu", "seq", "pos", "slots", "ws"))}
    if null:
        at[null] = None
    if off:
        at[off] += 2
    pool = lib.duo_block_pool(at["table"], at["free"], at["count"], at["lens"], batch, planes, block_size, max_blocks,
                              num_blocks)
    m = lib.duo_slot_map(at["cu"], at["seq"], at["pos"], at["slots"])
    p = lambda n: c_void_p(at[n])
    return lib.library().duo_block_tables_update(byref(pool), p("new"), max_tokens, p("lens_out"), p("count_out"),
                                                 byref(m), p("ws"), ws, None)


@pytest.mark.parametrize("args,status", [
    (dict(batch=0), 1), (dict(batch=65536), 1), (dict(planes=0), 1), (dict(planes=129), 1), (dict(block_size=0), 1),
    (dict(max_blocks=0), 1), (dict(num_blocks=0), 1), (dict(num_blocks=1 << 31), 1), (dict(max_tokens=-1), 1),
    (dict(block_size=1 << 16, max_blocks=1 << 15), 2), (dict(batch=65535, planes=128, max_blocks=257), 2),
    (dict(ws=8), 6), (dict(null="ws"), 6), (dict(off="ws"), 1),
] + [(dict(null=n), 1) for n in ("table", "free", "count", "lens", "new", "lens_out", "count_out", "cu", "seq", "pos",
                                  "slots")] + [(dict(off=n), 1) for n in ("table", "new", "cu", "slots")])
def test_block_tables_refusals(lib, args, status):
    assert _tables_call(lib, **args) == status
    assert lib.duo_last_error() != ""


def test_block_tables_workspace_size(lib):
    assert lib.duo_block_tables_workspace_size(0) == 0 and lib.duo_block_tables_workspace_size(-3) == 0
    sizes = [lib.duo_block_tables_workspace_size(b) for b in (1, 2, 1000, 65535)]
    assert sizes == sorted(sizes) and all(s % 16 == 0 and s > 0 for s in sizes)


def test_kv8_entry_points_refuse_a_null_handle(lib):
    cache, kv8, paged, m = lib.duo_kv_cache(), lib.duo_kv8_cache(), lib.duo_paged(), lib.duo_slot_map()
    calls = [lambda: lib.duo_kv_append_kv8(None, cache, kv8, None, None, 1, stream=0),
             lambda: lib.duo_kv_append_kv8_paged(None, cache, paged, kv8, None, None, 1, stream=0),
             lambda: lib.duo_kv_append_kv8_ragged(None, cache, paged, kv8, m, 1, None, None, stream=0),
             lambda: lib.duo_attn_decode_kv8(None, cache, kv8, None, None, None, stream=0),
             lambda: lib.duo_attn_decode_kv8_paged(None, cache, paged, kv8, None, None, None, stream=0),
             lambda: lib.duo_attn_decode_kv8_varlen(None, cache, None, kv8, None, 1, None, None, None, stream=0)]
    for call in calls:
        with pytest.raises(lib.DuoError, match="DUO_ERR_INVALID_ARG"):
            call()


def test_kv8_prefill_entry_points_refuse_a_null_handle(lib):
    cache, kv8, paged = lib.duo_kv_cache(), lib.duo_kv8_cache(), lib.duo_paged()
    calls = [lambda: lib.duo_attn_prefill_kv8(None, cache, kv8, None, None, None, 1, None, None, stream=0),
             lambda: lib.duo_attn_prefill_kv8_paged(None, cache, paged, kv8, None, None, None, 1, None, None, stream=0)]
    for call in calls:
        with pytest.raises(lib.DuoError, match="DUO_ERR_INVALID_ARG"):
            call()
    assert lib.duo_prefill_kv8_workspace_size(None, 1000, 16) == 0
