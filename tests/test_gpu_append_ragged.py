"""Packed appends into bf16 paged caches, with and without the rotation on the way."""

import numpy as np
import pytest
import torch

from kv8_util import check
from ragged_util import f64, kinds_of, normal, rotated, scattered_table, slot_map, slot_of

pytestmark = pytest.mark.gpu
CANARY = 5.0
BUFFERS = ("k_full", "v_full", "k_sr", "v_sr")


def _layer(rng, B, Hq, Hkv, D, S, R, kinds, page, cap):
    from streaming_kv_cache_duo_gb300 import DuoPagedLayer
    mb = -(-cap // page)
    table, nb = scattered_table(rng, B, max(1, sum(kinds)), mb)
    layer = DuoPagedLayer(B, Hq, Hkv, D, S, R, page, mb, nb, table if sum(kinds) else None, kinds)
    for name in BUFFERS:
        getattr(layer, name).fill_(CANARY)
    return layer, (table if sum(kinds) else None)


def _rows(layer, name, b, h, pos):
    """Row of position pos of head h of sequence b in the cache."""
    idx = layer.kind_index[h]
    if layer.is_retrieval[h]:
        t = layer.block_table[b, idx, pos // layer.block_size].item()
        return getattr(layer, name + "_full")[t, pos % layer.block_size]
    return getattr(layer, name + "_sr")[b, idx, slot_of(pos, layer.S, layer.R)]


@pytest.mark.parametrize("B,Hq,Hkv,n_ret,D,S,R,page,new,start,rd,layout", [
    (1, 4, 4, 2, 64, 4, 32, 128, [1], [0], 64, "half"),
    (5, 8, 4, 1, 128, 3, 20, 128, [1, 1, 0, 1, 1], [0, 130, 7, 2000, 23], 128, "interleaved"),
    (3, 8, 8, 8, 64, 4, 32, 256, [300, 1, 37], [255, 0, 100], 32, "half"),
    (4, 2, 2, 0, 128, 64, 100, 128, [150, 0, 1, 500], [0, 9, 63, 700], 96, "half"),
    (6, 16, 2, 1, 128, 0, 1, 128, [40, 3, 1, 129, 1, 2], [1, 0, 5, 127, 128, 600], 16, "interleaved"),
])
@pytest.mark.parametrize("rope", [True, False], ids=["rotated", "plain"])
def test_append(B, Hq, Hkv, n_ret, D, S, R, page, new, start, rd, layout, rope):
    from streaming_kv_cache_duo_gb300 import DuoRope, duo_device_error
    rng = np.random.default_rng(B * 7 + D + rd)
    kinds = kinds_of(Hkv, n_ret)
    layer, table = _layer(rng, B, Hq, Hkv, D, S, R, kinds, page, max(s + n for s, n in zip(start, new)))
    m = slot_map(table, page, start, new)
    N = sum(new)
    xt, x = normal(rng, N, Hq + 2 * Hkv, D)
    q, k, v = xt.cuda().split([Hq, Hkv, Hkv], 1)
    before = {name: getattr(layer, name).clone() for name in BUFFERS}
    r = DuoRope(D, rotary_dim=rd, layout=layout, scaling=dict(kind="yarn", factor=4.0, original=512)) if rope else None
    qo = layer.append_ragged(k, v, m, rope=r, q=q if rope else None)
    torch.cuda.synchronize()
    assert duo_device_error() == 0 and layer.n == 0
    pos = m.token_pos.cpu().numpy()
    if rope:
        y, tol = rotated(x, pos, r.inv_freq, rd, layout, r.scale)
        check(f64(qo), y[:, :Hq], tol[:, :Hq], "q")
    else:
        assert qo is None
        y, tol = x, np.zeros_like(x)
    held = np.full((B, S + R), -1)
    at = 0
    for b in range(B):
        for t in range(new[b]):
            p = start[b] + t
            kept = p < S or p >= start[b] + new[b] - R
            for h in range(Hkv):
                if kinds[h] or kept:
                    check(f64(_rows(layer, "k", b, h, p)), y[at + t, Hq + h], tol[at + t, Hq + h], f"k {b} {h} {p}")
                    assert torch.equal(_rows(layer, "v", b, h, p), v[at + t, h])
            if kept:
                held[b, slot_of(p, S, R)] = p
        at += new[b]
    if n_ret < Hkv:
        assert np.array_equal(layer.pos.cpu().numpy(), held)
    # nothing else was written: put back what was and compare
    for b in range(B):
        for t in range(new[b]):
            for h in range(Hkv):
                for name in ("k", "v"):
                    _rows(layer, name, b, h, start[b] + t).fill_(CANARY)
    for name in BUFFERS:
        assert torch.equal(getattr(layer, name), before[name]), name


def test_turned_down_and_padding_tokens_are_skipped():
    from streaming_kv_cache_duo_gb300 import DuoRope, duo_device_error
    rng = np.random.default_rng(1)
    layer, table = _layer(rng, 3, 4, 2, 64, 4, 32, [1, 0], 128, 300)
    m = slot_map(table, 128, [5, None, 200], [3, 4, 2], pad=6)
    N = 15
    q, k = (torch.ones(N, h, 64, dtype=torch.bfloat16, device="cuda") for h in (4, 2))
    out = torch.full_like(q, 9.0)
    layer.append_ragged(k, k, m, rope=DuoRope(64), q=q, q_out=out)
    torch.cuda.synchronize()
    assert duo_device_error() == 0
    assert (out[3:7] == 9).all() and (out[9:] == 9).all() and not (out[:3] == 9).any()
    assert (layer.pos[1] == -1).all() and (layer.k_sr[1] == CANARY).all()
    assert (layer.v_full == 1).all(-1).sum().item() == 5


@pytest.mark.parametrize("bad", ["slot", "negative", "sequence", "first", "last"])
def test_map_entries_out_of_range_are_not_dereferenced(bad):
    from streaming_kv_cache_duo_gb300 import DuoError, duo_device_error, _lib
    import ctypes
    rng = np.random.default_rng(2)
    layer, table = _layer(rng, 2, 2, 2, 64, 4, 32, [1, 0], 128, 300)
    m = slot_map(table, 128, [5, 40], [3, 4])
    if bad == "slot":
        m.slots[1, 0] = layer.k_full.shape[0] * 128
    elif bad == "negative":
        m.slots[1, 0] = -5
    elif bad == "sequence":
        m.token_seq[1] = 2
    elif bad == "first":
        m.cu_new[0] = 2
    else:
        m.cu_new[1] = 100
    k = torch.ones(7, 2, 64, dtype=torch.bfloat16, device="cuda")
    layer.append_ragged(k, k, m)
    code = ctypes.c_uint32()
    assert _lib.library().duo_device_error(ctypes.byref(code)) == _lib.DUO_ERR_INVALID_ARG
    # the rows that stay: all but those of the bad entries
    lost = {"slot": 1, "negative": 1, "sequence": 1, "first": 2, "last": 7}[bad]  # ("last" is also where sequence 1 begins)
    assert (layer.v_full == 1).all(-1).sum().item() == 7 - lost
    assert duo_device_error() == 0


def test_rows_past_4gb_of_pool():
    """A pool of more than 2^31 elements: rows at its end."""
    from streaming_kv_cache_duo_gb300 import DuoPagedLayer, duo_device_error
    nb, page, D = (1 << 31) // (128 * 128) + 5, 128, 128
    table = torch.tensor([[[nb - 1]]], dtype=torch.int32, device="cuda")
    layer = DuoPagedLayer(1, 1, 1, D, 4, 32, page, 1, nb, table, [1])
    m = slot_map(table, page, [100], [1])
    x = torch.randn(1, 1, D, device="cuda").to(torch.bfloat16)
    layer.append_ragged(x, -x, m)
    assert torch.equal(layer.k_full[nb - 1, 100], x[0, 0]) and torch.equal(layer.v_full[nb - 1, 100], -x[0, 0])
    assert duo_device_error() == 0


def test_refusals():
    from streaming_kv_cache_duo_gb300 import DuoError, DuoRope
    rng = np.random.default_rng(3)
    layer, table = _layer(rng, 2, 4, 2, 64, 4, 32, [1, 0], 128, 300)
    m = slot_map(table, 128, [5, 40], [3, 4])
    k = torch.ones(7, 2, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.ones(7, 4, 64, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: layer.append_ragged(k[:6], k[:6], m), lambda: layer.append_ragged(k, k.float(), m),
                 lambda: layer.append_ragged(k, k[:, :1], m), lambda: layer.append_ragged(k, k, m, rope=DuoRope(128)),
                 lambda: layer.append_ragged(k, k, m, rope=DuoRope(64), q=k),
                 lambda: layer.append_ragged(k, k, slot_map(table[:1], 128, [5], [7]))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(DuoError, match="DUO_ERR_INVALID_ARG"):
        layer.append_ragged(k, k, m, q=q)  # q without a rotation
    layer.paged.stream_table = layer.paged.block_table
    with pytest.raises(DuoError, match="DUO_ERR_UNSUPPORTED"):
        layer.append_ragged(k, k, m)
    assert (layer.k_full == CANARY).all()
