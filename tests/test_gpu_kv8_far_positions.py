"""Packed appends at the far end of the positions: the last that there is, and maps that pass it."""

import numpy as np
import pytest
import torch

from kv8_util import BLOCK

pytestmark = pytest.mark.gpu

PAGE, D, S, R, CANARY = 128, 64, 4, 32, 77
TOP = 2 ** 31 - 2  # the last position (a length has to stay below 2^31)


def _layer():
    from streaming_kv_cache_duo_gb300 import DuoKv8PagedLayer
    table = torch.zeros((3, 1, 2), dtype=torch.int32, device="cuda")  # (appends by map do not read it)
    layer = DuoKv8PagedLayer(3, 2, 2, D, S, R, PAGE, 2, 6, table, [1, 0])
    for name in ("k_codes", "v_codes", "k_scale", "v_scale", "k_tail", "v_tail", "k_sr", "v_sr"):
        getattr(layer, name).view(torch.uint8).fill_(CANARY)
    layer.pos.fill_(CANARY)
    return layer


def _append(layer, starts, counts):
    """counts[b] tokens of sequence b from position starts[b] on; positions past int32 wrap, as a
    caller's 32-bit sum would."""
    from streaming_kv_cache_duo_gb300 import DuoSlotMap
    at = np.concatenate([np.arange(s, s + c, dtype=np.int64) for s, c in zip(starts, counts)])
    seq = np.repeat(np.arange(3), counts)
    slots = 2 * seq * PAGE + at % (2 * PAGE)  # sequence b owns blocks 2 b and 2 b + 1
    dev = lambda a, t: torch.from_numpy(np.ascontiguousarray(a.astype(t))).cuda()
    m = DuoSlotMap(dev(np.concatenate([[0], np.cumsum(counts)]), np.int32), dev(seq, np.int32),
                   dev(at, np.int32), dev(slots, np.int64)[:, None].contiguous())
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(len(at), 2, D, generator=g).bfloat16().cuda() for _ in range(2))
    layer.append_ragged(k, v, m)
    return k, v


def _state(layer, b):
    """Everything that belongs to sequence b."""
    pool = lambda t: t[2 * b:2 * b + 2]
    parts = [pool(layer.k_codes), pool(layer.v_codes), pool(layer.k_scale), pool(layer.v_scale), layer.k_tail[b],
             layer.v_tail[b], layer.k_sr[b], layer.v_sr[b], layer.pos[b]]
    return [t.contiguous().view(torch.uint8).cpu() for t in parts]


def test_the_last_position_is_stored():
    from streaming_kv_cache_duo_gb300 import duo_device_error
    layer = _layer()
    counts = [2, 0, 70]
    k, v = _append(layer, [TOP - 1, 0, TOP - 69], counts)
    assert duo_device_error() == 0
    rows = TOP % BLOCK + 1
    for name, x in (("k", k), ("v", v)):
        tail = getattr(layer, name + "_tail")
        assert torch.equal(tail[0, 0, rows - 2:rows], x[:2, 0])
        assert torch.equal(tail[2, 0, :rows], x[-rows:, 0])
        assert torch.equal(getattr(layer, name + "_sr")[2, 0, S + (TOP - S) % R], x[-1, 1])
    assert layer.pos[2].max().item() == TOP


@pytest.mark.parametrize("start,count", [(TOP - 99, 200), (TOP - 64, 66), (TOP, 2), (TOP - 1, 300), (TOP + 1, 1)])
def test_a_sequence_past_the_last_position_is_left_as_it_was(start, count):
    from streaming_kv_cache_duo_gb300 import duo_device_error
    layer = _layer()
    before = _state(layer, 1)
    k, _ = _append(layer, [0, start, 5], [3, count, 3])
    assert duo_device_error() == 1 << 21
    assert all(torch.equal(a, b) for a, b in zip(_state(layer, 1), before))
    # its neighbours are stored all the same, and nothing of theirs but their rows is touched
    assert torch.equal(layer.k_tail[0, 0, :3], k[:3, 0]) and torch.equal(layer.k_tail[2, 0, 5:8], k[-3:, 0])
    raw = layer.k_tail.view(torch.uint8)
    assert (raw[0, 0, 3:] == CANARY).all() and (raw[2, 0, :5] == CANARY).all() and (raw[2, 0, 8:] == CANARY).all()
