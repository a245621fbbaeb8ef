"""8-bit caches over randomly drawn shapes: prefill a chunk, append it, decode, in every layout, each
against the oracle; and pools whose rows lie past 32-bit byte offsets."""

import numpy as np
import pytest
import torch

from kv8_util import BLOCK, Batch, attend, check, f64, scattered_table

pytestmark = pytest.mark.gpu


def _layer(c, cap, page, rng):
    from streaming_kv_cache_duo_gb300 import DuoKv8Layer, DuoKv8PagedLayer
    if page:
        mb = -(-cap // page)
        table, nb = scattered_table(rng, c.B, max(1, len(c.ret)), mb)
        table = table if c.ret else None
        return DuoKv8PagedLayer(c.B, c.Hq, c.Hkv, c.D, c.S, c.R, page, mb, nb, table, c.kinds, code=c.code)
    return DuoKv8Layer(c.B, c.Hq, c.Hkv, c.D, c.S, c.R, cap, c.kinds, code=c.code)


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(seed):
    from streaming_kv_cache_duo_gb300 import duo_device_error
    rng = np.random.default_rng(1000 + seed)
    D = int(rng.choice([64, 128]))
    Hkv = int(rng.choice([1, 2, 3, 5]))
    g = int(rng.choice([1, 2, 4, 8]))
    kinds = [int(x) for x in rng.integers(0, 2, Hkv)]
    S = int(rng.choice([0, 1, 4, 64, 130]))
    R = int(rng.choice([1, 5, 32, 127, 256, 300]))
    B = int(rng.integers(1, 4))
    n = int(rng.choice([0, 1, 60, 64, 200, 513, 1500]))
    T = int(rng.choice([1, 2, 63, 65, 130, 260]))
    page = int(rng.choice([0, 128, 256, 640]))
    code = str(rng.choice(["int8", "e4m3"]))
    what = dict(D=D, Hkv=Hkv, g=g, kinds=kinds, S=S, R=R, B=B, n=n, T=T, page=page, code=code)
    c = Batch(seed, [n + T] * B, Hkv * g, Hkv, D, S, R, kinds, code)
    layer = _layer(c, n + T, page, rng)
    cut = lambda x, a, b: x[:, a:b].contiguous().cuda()
    at = 0
    while at < n:
        step = int(rng.integers(1, n - at + 1))
        layer.append(cut(c.kt, at, at + step), cut(c.vt, at, at + step))
        at += step
    out = layer.prefill(cut(c.qt, n, n + T), cut(c.kt, n, n + T), cut(c.vt, n, n + T))
    layer.append(cut(c.kt, n, n + T), cut(c.vt, n, n + T))
    dec = layer.decode(c.query([n + T] * B))
    lens = torch.full((B,), n + T, dtype=torch.int32, device="cuda")
    assert torch.equal(layer.decode_varlen(c.query([n + T] * B), lens, n + T), dec), what
    torch.cuda.synchronize()
    assert duo_device_error() == 0, what
    got, gd = f64(out), f64(dec)
    rows = sorted({0, T // 2, T - 1})
    pos = np.arange(n + T)
    for b in range(B):
        ref, tol = c.decode(b, n + T)
        check(gd[b], ref, tol, f"decode {what}")
        for h in range(Hkv):
            kv = []
            for x in (c.k, c.v):
                held = c.heads_rows(b, h, n, x)[1]
                kv.append(np.concatenate([held, x[b, n:n + T, h]]))
            for t in rows:
                i = n + t
                see = pos <= i if kinds[h] else (pos <= i) & ((pos < S) | (i - pos < R))
                for j in range(h * g, h * g + g):
                    ref, tol = attend(c.q[b, i, j], kv[0][see], kv[1][see])
                    check(got[b, t, j], ref, tol, f"prefill row {t} head {j} {what}")


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_pools_past_four_gigabytes(code):
    """Blocks at the far end of a pool of 2^25 rows of 128 bytes and more."""
    from streaming_kv_cache_duo_gb300 import DuoKv8PagedLayer, duo_device_error
    n, page, nb = 700, 128, (1 << 18) + 9
    c = Batch(60, [n], 4, 1, 128, 4, 32, [1], code)
    ids = [nb - 1, nb - 3, 0, nb - 2, 7, nb - 4]
    table = torch.tensor(ids, dtype=torch.int32, device="cuda").reshape(1, 1, -1)
    layer = DuoKv8PagedLayer(1, 4, 1, 128, 4, 32, page, len(ids), nb, table, [1], code=code)
    c.fill(layer, 333)
    ref, tol = c.decode(0, n)
    check(f64(layer.decode(c.query([n])))[0], ref, tol)
    cut = lambda x: x[:, :5].contiguous().cuda()
    layer.prefill(cut(c.qt), cut(c.kt), cut(c.vt))
    torch.cuda.synchronize()
    assert duo_device_error() == 0
    used = layer.k_codes.view(torch.uint8)[torch.tensor(ids, device="cuda").long()]
    assert bool(used[:5].any(-1).all())  # five blocks of full rows
    assert layer.k_codes.view(torch.uint8)[1:6].max().item() == 0  # and nowhere else


def test_slots_past_two_to_the_31():
    from streaming_kv_cache_duo_gb300 import DuoBlockPool, duo_device_error
    from oracle.kv8 import block_tables_update
    nb, bs = 1 << 20, 4096
    pool = DuoBlockPool(2, 1, bs, 5, nb, 64)
    new = [40, 20]
    want = block_tables_update(pool.block_table.cpu().numpy(), pool.free_list.cpu().numpy(), nb, [0, 0], new, bs, 64)
    m = pool.update(torch.tensor(new, dtype=torch.int32, device="cuda"))
    assert duo_device_error() == 0
    assert np.array_equal(m.slots.cpu().numpy(), want["slots"]) and want["slots"].max() > 1 << 31
