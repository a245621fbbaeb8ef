"""Block tables, slot maps and the free list built on the device equal the sequential oracle, for
any batch; capture in a CUDA graph; what is turned down; what is refused."""

import numpy as np
import pytest
import torch

from oracle.kv8 import block_tables_update

pytestmark = pytest.mark.gpu


def _pool(B, planes, bs, mb, nb, N):
    from streaming_kv_cache_duo_gb300 import DuoBlockPool
    return DuoBlockPool(B, planes, bs, mb, nb, N)


def _state(pool):
    return (pool.block_table.cpu().numpy(), pool.free_list.cpu().numpy(), int(pool.free_count), pool.seq_lens.cpu().numpy())


def _same(pool, want, lens=None, count=None):
    live = want["free_count"]
    assert int(pool.free_count if count is None else count) == live
    assert np.array_equal((pool.seq_lens if lens is None else lens).cpu().numpy(), want["seq_lens"])
    assert np.array_equal(pool.block_table.cpu().numpy(), want["block_table"])
    assert np.array_equal(pool.free_list.cpu().numpy(), want["free_list"])
    for name in ("cu_new", "token_seq", "token_pos", "slots"):
        assert np.array_equal(getattr(pool.slot_map, name).cpu().numpy(), want[name]), name


def _step(pool, new, bs):
    want = block_tables_update(*_state(pool), new, bs, pool.max_tokens)
    pool.update(torch.tensor(new, dtype=torch.int32, device="cuda"))
    return want


CASES = [
    # B, planes, block size, max_blocks, num_blocks, max_tokens, most new tokens, steps
    (1, 1, 128, 3, 3, 1, 1, 5),
    (3, 2, 4, 6, 40, 16, 6, 30),
    (70, 3, 128, 9, 2000, 4000, 200, 12),
    (1500, 2, 16, 4, 9000, 9000, 9, 8),   # more sequences than scanning threads, two launches
    (5, 8, 1, 40, 1700, 3000, 35, 8),     # blocks of one token
    (2, 1, 384, 50, 100, 20000, 9000, 4),
]


@pytest.mark.parametrize("case", CASES, ids=[f"case{i}" for i in range(len(CASES))])
def test_steps_match_the_oracle(case):
    from streaming_kv_cache_duo_gb300 import DuoError, duo_device_error
    B, planes, bs, mb, nb, N, most, steps = case
    rng = np.random.default_rng(20)
    pool = _pool(B, planes, bs, mb, nb, N)
    pool.free_list.copy_(torch.from_numpy(rng.permutation(nb).astype(np.int32)))
    for _ in range(steps):
        new = rng.integers(0, most + 1, B)
        new[rng.random(B) < 0.2] = -1
        want = _step(pool, new, bs)
        _same(pool, want)
        if want["turned_down"]:
            with pytest.raises(DuoError, match="DUO_ERR_CAPACITY"):
                _raise(duo_device_error)
        else:
            assert duo_device_error() == 0


def _raise(duo_device_error):
    """duo_device_error() returns the code; the status behind it goes with the message."""
    from streaming_kv_cache_duo_gb300 import DuoError, _lib
    import ctypes
    code = ctypes.c_uint32()
    st = _lib.library().duo_device_error(ctypes.byref(code))
    assert code.value != 0 or st == 0
    if st:
        raise DuoError(st, _lib.duo_last_error())


def test_separate_outputs_leave_the_inputs_and_repeat():
    rng = np.random.default_rng(21)
    pool = _pool(8, 2, 16, 10, 200, 300)
    _step(pool, rng.integers(1, 100, 8) // 4, 16)
    lens, count = torch.empty_like(pool.seq_lens), torch.empty_like(pool.free_count)
    new = rng.integers(0, 60, 8) // 2
    new[3] = -1
    before = _state(pool)
    want = block_tables_update(*before, new, 16, pool.max_tokens)
    for _ in range(3):
        pool.update(torch.tensor(new, dtype=torch.int32, device="cuda"), seq_lens_out=lens, free_count_out=count)
        _same(pool, want, lens, count)
        assert np.array_equal(pool.seq_lens.cpu().numpy(), before[3]) and int(pool.free_count) == before[2]


def test_sequences_past_the_tables_or_the_batch_are_turned_down():
    from streaming_kv_cache_duo_gb300 import DuoError, duo_device_error
    pool = _pool(4, 1, 8, 2, 20, 12)
    # sequence 1 would pass its table (16 tokens), 3 the packed batch (12 tokens)
    want = _step(pool, np.array([4, 17, 0, 5]), 8)
    assert want["turned_down"]
    _same(pool, want)
    with pytest.raises(DuoError, match="DUO_ERR_CAPACITY"):
        _raise(duo_device_error)


def test_bad_values_are_reported_and_stay_in_bounds():
    from streaming_kv_cache_duo_gb300 import DuoError, duo_device_error
    def fresh():
        pool = _pool(3, 2, 8, 4, 30, 24)
        _step(pool, np.array([9, 8, 3]), 8)
        return pool
    for what in ("length", "length_high", "new", "count", "count_high", "table", "free", "returned"):
        pool = fresh()
        new = torch.tensor([2, 2, 2], dtype=torch.int32, device="cuda")
        if what == "length":
            pool.seq_lens[1] = -4
        elif what == "length_high":
            pool.seq_lens[1] = 33
        elif what == "new":
            new[1] = -2
        elif what == "count":
            pool.free_count[0] = -1
        elif what == "count_high":
            pool.free_count[0] = 31
        elif what == "table":
            pool.block_table[0, 1, 1] = 30
        elif what == "free":
            pool.free_list[:] = -7
            new[:] = 8
        else:
            pool.block_table[0, 1, 0] = -1
            new[:] = 0
            new[0] = -1
        free0 = int(pool.free_count)
        pool.update(new)
        with pytest.raises(DuoError, match="DUO_ERR_INVALID_ARG"):
            _raise(duo_device_error)
        slots = pool.slot_map.slots.cpu().numpy()
        assert slots.min() >= -1 and slots.max() < 30 * 8
        if what in ("length", "length_high", "new"):
            assert (pool.slot_map.token_pos.cpu().numpy()[2:4] == ([-1, -1] if what != "new" else [3, 4])).all()
        if what == "returned":  # three good ids of four came back
            assert int(pool.free_count) == free0 + 3
    assert duo_device_error() == 0


def test_more_returns_than_blocks_stay_in_the_list():
    from streaming_kv_cache_duo_gb300 import DuoError, duo_device_error
    pool = _pool(2, 1, 8, 4, 8, 16)
    _step(pool, np.array([8, 8]), 8)
    pool.free_count[0] = 8  # as if the blocks had been freed already
    pool.update(torch.tensor([-1, -1], dtype=torch.int32, device="cuda"))
    assert int(pool.free_count) == 8
    with pytest.raises(DuoError, match="DUO_ERR_INVALID_ARG"):
        _raise(duo_device_error)


def test_capture_and_replay():
    rng = np.random.default_rng(22)
    pool = _pool(16, 2, 128, 20, 700, 64)
    _step(pool, rng.integers(0, 5, 16), 128)
    new = torch.zeros(16, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        pool.update(new)
    for step in range(4):
        vals = rng.integers(0, 5, 16)
        vals[step] = -1
        want = block_tables_update(*_state(pool), vals, 128, 64)
        new.copy_(torch.from_numpy(vals.astype(np.int32)))
        g.replay()
        torch.cuda.synchronize()
        _same(pool, want)


def test_refusals():
    pool = _pool(4, 2, 128, 8, 64, 32)
    from streaming_kv_cache_duo_gb300 import DuoError, _lib
    new = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (new[:3].contiguous(), new.long(), new.cpu(), torch.zeros(8, dtype=torch.int32, device="cuda")[::2]):
        with pytest.raises(ValueError):
            pool.update(bad)
    small = pool.workspace[:16]
    with pytest.raises(DuoError, match="DUO_ERR_WORKSPACE"):
        _lib.duo_block_tables_update(pool.c, new, 32, pool.seq_lens, pool.free_count, pool.slot_map.c, small)


def test_tables_serve_the_bf16_paged_caches():
    """The pool's table behind a bf16 paged layer, sequences of one length: the same rows as a
    contiguous layer's, so a prefill, appends and a decode give the same bits."""
    from streaming_kv_cache_duo_gb300 import DuoLayer, DuoPagedLayer
    B, Hq, Hkv, D, S, R, page, mb = 2, 4, 2, 64, 4, 32, 128, 3
    kinds, g = [1, 0], torch.Generator().manual_seed(3)
    pool = _pool(B, 1, page, mb, B * mb, B * 300)
    paged = DuoPagedLayer(B, Hq, Hkv, D, S, R, page, mb, B * mb, pool.block_table, kinds)
    plain = DuoLayer(B, Hq, Hkv, D, S, R, page * mb, kinds)
    paged.k_full.zero_(), paged.v_full.zero_()
    for T in (1, 127, 130, 1):
        q, k, v = (torch.randn(B, T, h, D, generator=g).bfloat16().cuda() for h in (Hq, Hkv, Hkv))
        pool.update(torch.full((B,), T, dtype=torch.int32, device="cuda"))
        assert torch.equal(paged.prefill(q, k, v), plain.prefill(q, k, v))
        paged.append(k, v)
        plain.append(k, v)
        last = q[:, -1].contiguous()
        a, b = paged.decode(last), plain.decode(last)
        assert torch.equal(a, b)
        n = paged.n
        for s in range(B):
            rows = paged.k_full[pool.block_table[s, 0, :-(-n // page)].long()].reshape(-1, D)[:n]
            assert torch.equal(rows, plain.k_full[s, 0, :n])
    assert int(pool.free_count) == 0 and pool.seq_lens.tolist() == [259, 259]
