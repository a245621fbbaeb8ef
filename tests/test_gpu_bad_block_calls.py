"""A block id outside the pool concerns the rows it names alone: the rest of the same call, and every
later call, computes what it would have computed without it, whether or not the error has been read."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def _rand(g, *shape):
    return torch.randn(*shape, generator=g).bfloat16().cuda()


@pytest.mark.parametrize("D,pool", [(64, False), (128, False), (128, True)])
def test_other_sequences_and_later_prefills_are_computed(D, pool):
    from streaming_kv_cache_duo_gb300 import DuoKv8Layer, DuoLayer, DuoPagedLayer, duo_device_error
    B, Hq, Hkv, S, R, page, mb, n, T = 2, 4, 2, 4, 32, 128, 4, 300, 40
    kinds, g = [1, 0], torch.Generator().manual_seed(11)
    ids = torch.randperm(2 * B * mb, generator=g).int()
    table, stream = ids[:B * mb].reshape(B, 1, mb).cuda(), ids[B * mb:].reshape(B, 1, mb).cuda()
    paged = DuoPagedLayer(B, Hq, Hkv, D, S, R, page, mb, 2 * B * mb, table, kinds, stream_table=stream if pool else None)
    plain = DuoLayer(B, Hq, Hkv, D, S, R, page * mb, kinds)
    kv8 = DuoKv8Layer(B, Hq, Hkv, D, S, R, page * mb, kinds)
    k, v = _rand(g, B, n, Hkv, D), _rand(g, B, n, Hkv, D)
    paged.k_full.zero_(), paged.v_full.zero_()
    for layer in (paged, plain, kv8):
        layer.append(k, v)
    q, k, v = _rand(g, B, T, Hq, D), _rand(g, B, T, Hkv, D), _rand(g, B, T, Hkv, D)
    want, want8, good = plain.prefill(q, k, v), kv8.prefill(q, k, v), paged.prefill(q, k, v)
    assert duo_device_error() == 0
    kept = table[0, 0, 1].item()
    table[0, 0, 1] = 10 ** 6
    mark = lambda: torch.full_like(q, 77.0)
    first, plain_out, kv8_out, again = mark(), mark(), mark(), mark()
    paged.prefill(q, k, v, out=first)
    table[0, 0, 1] = kept
    plain.prefill(q, k, v, out=plain_out)
    kv8.prefill(q, k, v, out=kv8_out)
    paged.prefill(q, k, v, out=again)
    torch.cuda.synchronize()
    assert duo_device_error() & (1 << 21)
    assert torch.equal(first[1], good[1])            # the other sequence
    assert torch.equal(first[0, :, 2:], good[0, :, 2:])  # the streaming head
    assert bool((first[0] != 77.0).any(-1).all())
    assert torch.equal(plain_out, want) and torch.equal(kv8_out, want8) and torch.equal(again, good)
    assert duo_device_error() == 0
