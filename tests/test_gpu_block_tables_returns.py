"""Thousands of blocks given back in one step, by small and large batches, with ids among them that are
none: the free list, counts and tables of the sequential oracle."""

import numpy as np
import pytest
import torch

from oracle.kv8 import block_tables_update

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [0, 9])
@pytest.mark.parametrize("B,planes,bs,mb,tokens", [(64, 8, 1, 128, 8192), (5, 128, 2, 60, 600), (1600, 2, 16, 4, 9000)])
def test_many_blocks_come_back(B, planes, bs, mb, tokens, bad):
    from streaming_kv_cache_duo_gb300 import DuoBlockPool, duo_device_error
    rng = np.random.default_rng(90)
    nb = B * planes * mb
    pool = DuoBlockPool(B, planes, bs, mb, nb, tokens)
    pool.free_list.copy_(torch.from_numpy(rng.permutation(nb).astype(np.int32)))

    def step(new):
        want = block_tables_update(pool.block_table.cpu().numpy(), pool.free_list.cpu().numpy(), int(pool.free_count),
                                   pool.seq_lens.cpu().numpy(), new, bs, tokens)
        pool.update(torch.from_numpy(new.astype(np.int32)).cuda())
        for name in ("seq_lens", "block_table", "free_list"):
            assert np.array_equal(getattr(pool, name).cpu().numpy(), want[name]), name
        assert int(pool.free_count) == want["free_count"]
        for name in ("cu_new", "token_seq", "token_pos", "slots"):
            assert np.array_equal(getattr(pool.slot_map, name).cpu().numpy(), want[name]), name

    step(np.full(B, min(tokens // B, bs * mb - 1)))
    assert duo_device_error() == 0
    new = np.full(B, -1)
    new[::7] = 1  # these go on, out of what the others gave back too
    if bad:
        gone = [b for b in range(B) if new[b] < 0]
        for i in range(bad):
            pool.block_table[gone[i * 5 % len(gone)], i % planes, 0] = [-1, nb, -7][i % 3]
    free0 = int(pool.free_count)
    step(new)
    assert (duo_device_error() == 0) == (bad == 0)
    assert int(pool.free_count) - free0 > 2 * 1024
    step(np.full(B, -1))
    assert duo_device_error() == 0
