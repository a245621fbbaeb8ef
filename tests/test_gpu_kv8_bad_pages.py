"""Pages of an 8-bit cache that do not exist: their rows are left out of the softmax, by the decode and
by the prefill alike, so both give the attention over the keys that are there."""

import numpy as np
import pytest
import torch

from kv8_util import Batch, attend, check, f64, scattered_table

pytestmark = pytest.mark.gpu
PAGE = 128


def _layer(c, cap):
    from streaming_kv_cache_duo_gb300 import DuoKv8PagedLayer
    mb = -(-cap // PAGE)
    table, nb = scattered_table(np.random.default_rng(3), c.B, len(c.ret), mb)
    return DuoKv8PagedLayer(c.B, c.Hq, c.Hkv, c.D, c.S, c.R, PAGE, mb, nb, table, c.kinds, code=c.code)


def _want(c, b, h, j, n, i, gone):
    """Output and bound of the query of head j at position i over n cached rows and the positions from
    n up to it, without the pages `gone` of a retrieval head's full blocks."""
    at = np.arange(i + 1)
    keep = {}
    for name, x in (("k", c.k), ("v", c.v)):
        keep[name] = np.concatenate([c.heads_rows(b, h, n, x)[1], x[b, n:i + 1, h]])
    if c.kinds[h]:
        see = ~(np.isin(at // PAGE, gone) & (at < n // 64 * 64))
    else:
        see = (at < c.S) | (i - at < c.R)
    return attend(c.q[b, i, j], keep["k"][see], keep["v"][see])


CASES = [
    # D, n, T, gone: a split item; whole items; a page with nothing but the open block (which is in the tail,
    # so nobody reads the page); all pages; half a tile
    (64, 1000, 5, [2]), (128, 400, 300, [0]), (128, 700, 64, [5]), (64, 384, 20, [0, 1, 2]), (128, 192, 7, [1]),
    (128, 5000, 30, [0, 3, 4, 5, 6, 7, 20, 38]),
]


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("D,n,T,gone", CASES)
def test_rows_of_missing_pages_are_left_out(D, n, T, gone, code):
    from streaming_kv_cache_duo_gb300 import duo_device_error
    c = Batch(70, [n + T] * 2, 8, 2, D, 4, 32, [1, 0], code, scale=1.5)
    layer = _layer(c, n + T)
    layer.append(c.kt[:, :n].contiguous().cuda(), c.vt[:, :n].contiguous().cuda())
    assert duo_device_error() == 0
    for page, bad in zip(gone, (-1, layer.k_codes.shape[0], 0x7fffffff, -(1 << 31)) * 2):
        layer.block_table[0, 0, page] = bad
    pick = lambda x: x[:, n:n + T].contiguous().cuda()
    got = f64(layer.prefill(pick(c.qt), pick(c.kt), pick(c.vt)))
    error = 1 << 21 if min(gone) * PAGE < n // 64 * 64 else 0
    assert duo_device_error() == error
    dec = f64(layer.decode(c.query([n, n])))
    assert duo_device_error() == error
    for b in range(2):
        for h in range(2):
            for j in range(h * 4, h * 4 + 4):
                lost = gone if b == 0 else []
                for t in sorted({0, T // 2, T - 1}):
                    check(got[b, t, j], *_want(c, b, h, j, n, n + t, lost), f"prefill {b} {t} {j}")
                ref = _want(c, b, h, j, n, n - 1, lost)
                check(dec[b, j], *ref, f"decode {b} {j}")
