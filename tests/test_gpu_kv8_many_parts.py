"""Decodes over 8-bit caches whose units are split over more CTAs than the merge takes in one pass, with
the key that counts most in a part of the first and of the last pass; workspaces of exactly the size
asked for; contiguous caches with lengths on the device; calls repeated."""

import numpy as np
import pytest
import torch

from kv8_util import BLOCK, Batch, attend, check, f64, ring, scattered_table

pytestmark = pytest.mark.gpu


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _parts(B, n_ret, n_str, g, D, n, SR, code):
    """(parts per retrieval unit, parts the merge takes in one pass) as the decode plans them: tiles of 256
    keys (512 at D = 64) and one for the tail, one more place a unit, shared out over the SMs; the wide merge
    (few units: 32 dims of a head per CTA) takes 4 x 20 parts a pass, the other 8 / g x 4."""
    tile = 256 if D == 128 else 512
    tiles = -(-(n // BLOCK * BLOCK) // tile) + (n % BLOCK > 0)
    ring_tiles = -(-min(n, SR) // 128)
    U_r, U_s = B * n_ret, B * n_str
    weight = 8 * U_r * (tiles + 1) + (7 if code == "int8" and SR > 128 else 8) * U_s * (ring_tiles + 1)
    C = min(_sms(), weight // 20)
    U = U_r + U_s
    wide = U <= C and U * g * (D // 32) <= _sms()
    return 8 * (tiles + 1) * C // weight, 80 if wide else 8 // g * 4


def _paged(c, lens, cap, rng):
    from streaming_kv_cache_duo_gb300 import DuoBlockPool, DuoKv8PagedLayer
    mb = -(-(cap + 1) // 128)
    pool = DuoBlockPool(c.B, len(c.ret), 128, mb, c.B * len(c.ret) * mb, int(sum(lens)))
    layer = DuoKv8PagedLayer(c.B, c.Hq, c.Hkv, c.D, c.S, c.R, 128, mb, c.B * len(c.ret) * mb, pool.block_table, c.kinds,
                             code=c.code)
    m = pool.update(torch.tensor([int(n) for n in lens], dtype=torch.int32, device="cuda"))
    layer.append_ragged(*c.packed([0] * c.B, [int(n) for n in lens]), m)
    return layer


def _flat(c, cap):
    from streaming_kv_cache_duo_gb300 import DuoKv8Layer
    return DuoKv8Layer(c.B, c.Hq, c.Hkv, c.D, c.S, c.R, cap, c.kinds, code=c.code)


def _aim(c, b, n, h, at):
    """Makes the key at position `at` of head h the one that most of the weight of its first query head goes
    to: k along q, with a score a little above the logarithm of the number of keys."""
    q = c.q[b, n - 1, h * c.g]
    k = q * (np.log(n) + 2.0) * np.sqrt(c.D) / (q @ q)
    c.kt[b, at, h] = torch.from_numpy(k.astype(np.float32)).bfloat16()
    c.k[b, at, h] = c.kt[b, at, h].double().numpy()


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("place", [0.004, 0.93])
@pytest.mark.parametrize("g", [1, 2])
def test_one_unit_over_all_sms(g, place, code):
    n = 100_003
    parts, once = _parts(1, 1, 0, g, 128, n, 36, code)
    assert once == 80 and parts > once and int(place * parts) // once == (place > 0.5)
    c = Batch(80, [n], g, 1, 128, 4, 32, [1], code)
    _aim(c, 0, n, 0, int(place * n))
    layer = _flat(c, n)
    c.fill(layer)
    got = f64(layer.decode(c.query([n])))
    check(got[0], *c.decode(0, n))


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("B,Hq,Hkv,kinds,D,n", [(8, 12, 3, [1, 0, 1], 128, 16_411), (3, 16, 2, [1, 1], 128, 12_070),
                                               (5, 16, 2, [1, 1], 64, 20_000)])
def test_many_units_over_many_ctas_each(B, Hq, Hkv, kinds, D, n, ragged, code):
    from streaming_kv_cache_duo_gb300 import duo_device_error
    g = Hq // Hkv
    parts, once = _parts(B, sum(kinds), Hkv - sum(kinds), g, D, n, 36, code)
    assert once == 8 // g * 4 and parts > once
    lens = [n - 97 * b for b in range(B)] if ragged else [n] * B
    c = Batch(81, lens, Hq, Hkv, D, 4, 32, kinds, code)
    for b in range(B):  # the first and the last parts of a unit in turn
        for h in c.ret:
            _aim(c, b, lens[b], h, 70 if (b + h) % 2 else lens[b] - 130)
    q = c.query(lens)
    if ragged:
        layer = _paged(c, lens, n, np.random.default_rng(4))
        out = layer.decode_varlen(q, torch.tensor(lens, dtype=torch.int32, device="cuda"), n)
    else:
        layer = _flat(c, n)
        c.fill(layer)
        out = layer.decode(q)
    torch.cuda.synchronize()
    assert duo_device_error() == 0
    got = f64(out)
    for b in range(B):
        check(got[b], *c.decode(b, lens[b]), f"sequence {b}")


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("D,Hq,lens", [
    (128, 4, [0, 1, 63, 64, 65, 2000, 128, 700]), (64, 8, [1999, 64, 0, 5, 1300]), (64, 2, [40_000, 0, 1, 33_333]),
    (128, 16, [511] + [0, 64, 100] * 30),
])
def test_contiguous_caches_with_lengths_on_the_device(D, Hq, lens, code):
    """Each sequence's cache as it is at its own length: its open block in the tail, its ring."""
    from streaming_kv_cache_duo_gb300 import duo_device_error
    S, R, top = 4, 32, max(lens)
    c = Batch(82, [top] * len(lens), Hq, 2, D, S, R, [1, 0], code)
    layer = _flat(c, top)
    c.fill(layer)
    for name, t, x in (("k", c.kt, c.k), ("v", c.vt, c.v)):
        tail, sr = getattr(layer, name + "_tail"), getattr(layer, name + "_sr")
        tail.fill_(float("nan")), sr.fill_(float("nan"))
        for b, n in enumerate(lens):
            tail[b, 0, :n % BLOCK] = t[b, n // BLOCK * BLOCK:n, 0].cuda()
            pos, rows = ring(x[b, :n, 1], S, R)
            sr[b, 0, torch.from_numpy(pos >= 0).cuda()] = torch.from_numpy(rows[pos >= 0]).bfloat16().cuda()
            layer.pos[b] = torch.from_numpy(pos.astype(np.int32)).cuda()
    out = layer.decode_varlen(c.query(lens), torch.tensor(lens, dtype=torch.int32, device="cuda"), top)
    torch.cuda.synchronize()
    assert duo_device_error() == 0
    got = f64(out)
    for b, n in enumerate(lens):
        check(got[b], *c.decode(b, n), f"sequence {b} of {n} tokens")


@pytest.mark.parametrize("B,Hq,Hkv,kinds,D,n", [
    (1, 1, 1, [1], 64, 50_000),      # one unit: merge jobs by unit
    (1, 8, 1, [1], 128, 30_000), (1, 8, 8, [1] * 8, 128, 9000), (20, 8, 1, [1], 64, 3000), (200, 2, 2, [1, 0], 64, 700),
])
def test_a_workspace_of_the_size_asked_for_is_enough(B, Hq, Hkv, kinds, D, n):
    from streaming_kv_cache_duo_gb300 import _lib
    c = Batch(83, [n] * B, Hq, Hkv, D, 4, 32, kinds, "int8")
    layer = _flat(c, n)
    c.fill(layer)
    q = c.query([n] * B)
    want = layer.decode(q)
    size = _lib.duo_decode_workspace_size(layer.handle, n)
    ws = torch.full((size + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    for device_lens in (False, True):
        out = torch.full_like(q, 7.0)
        if device_lens:
            _lib.duo_attn_decode_kv8_varlen(layer.handle, layer.cache, None, layer.kv8, lens, n, q, out, ws[:size])
        else:
            _lib.duo_attn_decode_kv8(layer.handle, layer.cache, layer.kv8, q, out, ws[:size])
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert bool((ws[size:] == 0x5A).all())


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_calls_repeat_themselves_bit_for_bit(code):
    """Decodes and prefills, split and merged, give the same bits each time."""
    n, T = 21_000, 40
    c = Batch(84, [n + T] * 2, 8, 2, 128, 4, 200, [1, 0], code)
    layer = _flat(c, n + T)
    layer.append(c.kt[:, :n].contiguous().cuda(), c.vt[:, :n].contiguous().cuda())
    q = c.query([n, n])
    lens = torch.tensor([n, n - n % BLOCK], dtype=torch.int32, device="cuda")
    qs, k, v = (x[:, n:].contiguous().cuda() for x in (c.qt, c.kt, c.vt))
    one = lambda: (layer.decode(q), layer.decode_varlen(q, lens, n), layer.prefill(qs, k, v))
    first = one()
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(first, one()))


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("B,n,T,page,kinds", [(5, 130, 20, 0, [1, 0]), (6, 700, 64, 128, [1, 0]), (17, 300, 5, 128, [0, 1]),
                                              (9, 1000, 300, 0, [1, 1])])
def test_prefill_of_many_sequences(B, n, T, page, kinds, code):
    from streaming_kv_cache_duo_gb300 import DuoKv8PagedLayer, duo_device_error
    c = Batch(85, [n + T] * B, 4, 2, 64, 4, 32, kinds, code)
    if page:
        mb = -(-(n + T) // page)
        table, nb = scattered_table(np.random.default_rng(5), B, 1, mb)
        layer = DuoKv8PagedLayer(B, 4, 2, 64, 4, 32, page, mb, nb, table, kinds, code=code)
    else:
        layer = _flat(c, n + T)
    layer.append(c.kt[:, :n].contiguous().cuda(), c.vt[:, :n].contiguous().cuda())
    got = f64(layer.prefill(*(x[:, n:].contiguous().cuda() for x in (c.qt, c.kt, c.vt))))
    assert duo_device_error() == 0
    for b in range(B):
        for h in range(2):
            k, v = (np.concatenate([c.heads_rows(b, h, n, x)[1], x[b, n:, h]]) for x in (c.k, c.v))
            for t in (0, T // 2, T - 1):
                at, i = np.arange(n + T), n + t
                see = (at <= i) & (np.ones(n + T, bool) if kinds[h] else (at < 4) | (i - at < 32))
                for j in (2 * h, 2 * h + 1):
                    check(got[b, t, j], *attend(c.q[b, i, j], k[see], v[see]), f"sequence {b} row {t} head {j}")
