"""Prefill of a chunk against 8-bit caches: every head of sampled rows against attention in 64 bits
over the cache's rows (code * scale; the open block's as they were) and the chunk's own keys, within
the bound of kv8_util.attend."""

import numpy as np
import pytest
import torch

from kv8_util import BLOCK, Batch, attend, check, f64, scattered_table

pytestmark = pytest.mark.gpu


def _layer(c, cap, page=0, seed=1):
    from streaming_kv_cache_duo_gb300 import DuoKv8Layer, DuoKv8PagedLayer
    if page:
        mb = -(-cap // page)
        table, nb = scattered_table(np.random.default_rng(seed), c.B, len(c.ret), mb)
        return DuoKv8PagedLayer(c.B, c.Hq, c.Hkv, c.D, c.S, c.R, page, mb, nb, table, c.kinds, code=c.code)
    return DuoKv8Layer(c.B, c.Hq, c.Hkv, c.D, c.S, c.R, cap, c.kinds, code=c.code)


def _check_chunk(c, n, T, out, rows=None):
    got = f64(out)
    for b in range(c.B):
        for h in range(c.Hkv):
            keep = {}
            for name, x in (("k", c.k), ("v", c.v)):
                cached = c.heads_rows(b, h, n, x)[1]
                keep[name] = np.concatenate([cached, x[b, n:n + T, h]])
            at = np.arange(n + T)
            for t in rows if rows is not None else range(T):
                i = n + t
                see = at <= i
                if not c.kinds[h]:
                    see &= (at < c.S) | (i - at < c.R)
                for j in range(h * c.g, (h + 1) * c.g):
                    ref, tol = attend(c.q[b, i, j], keep["k"][see], keep["v"][see])
                    check(got[b, t, j], ref, tol, f"sequence {b} row {t} head {j}")


def _run(c, layer, n, T):
    from streaming_kv_cache_duo_gb300 import duo_device_error
    pick = lambda x: x[:, n:n + T].contiguous().cuda()
    out = layer.prefill(pick(c.qt), pick(c.kt), pick(c.vt))
    torch.cuda.synchronize()
    assert duo_device_error() == 0
    return out


def _fill(c, layer, n):
    if n:
        layer.append(c.kt[:, :n].contiguous().cuda(), c.vt[:, :n].contiguous().cuda())
        for name in ("k", "v"):  # nothing past the tokens may be used
            getattr(layer, name + "_tail")[:, :, n % BLOCK:] = float("nan")
            if layer.paged is None:
                getattr(layer, name + "_scale")[:, :, n // BLOCK:] = float("nan")


CASES = [
    # B, Hq, Hkv, D, S, R, kinds, n, T, page
    (1, 2, 2, 128, 4, 32, [1, 0], 0, 5, 0),
    (1, 2, 2, 128, 4, 32, [1, 0], 1, 1, 0),
    (2, 4, 2, 64, 4, 32, [1, 0], 63, 130, 0),
    (1, 4, 1, 128, 4, 32, [1], 64, 3, 0),
    (1, 4, 2, 128, 64, 256, [0, 1], 65, 300, 128),
    (1, 8, 1, 64, 4, 32, [1], 191, 40, 256),
    (2, 4, 2, 128, 0, 5, [1, 1], 128, 257, 0),
    (1, 4, 2, 128, 3, 100, [1, 0], 1000, 70, 384),
    (1, 2, 2, 64, 4, 32, [0, 0], 500, 33, 0),
    (1, 2, 1, 128, 4, 32, [1], 2500, 9, 128),
]


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("case", CASES, ids=[f"case{i}" for i in range(len(CASES))])
def test_chunks_match(case, code):
    B, Hq, Hkv, D, S, R, kinds, n, T, page = case
    c = Batch(50, [n + T] * B, Hq, Hkv, D, S, R, kinds, code)
    layer = _layer(c, n + T, page)
    _fill(c, layer, n)
    out = _run(c, layer, n, T)
    _check_chunk(c, n, T, out, None if T <= 40 else sorted({0, 1, T // 2, T - 2, T - 1, min(T - 1, 127), min(T - 1, 128)}))


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_a_chunked_prompt_then_decode(code):
    """Chunks of odd sizes, each prefilled then appended, and a decode over what they leave."""
    B, Hq, Hkv, D = 1, 8, 2, 128
    chunks = [200, 1, 319, 64, 77]
    c = Batch(51, [sum(chunks) + 1], Hq, Hkv, D, 4, 64, [1, 0], code)
    layer = _layer(c, sum(chunks) + 1, 128)
    n = 0
    for T in chunks:
        out = _run(c, layer, n, T)
        _check_chunk(c, n, T, out, sorted({0, T // 3, T - 1}))
        layer.append(c.kt[:, n:n + T].contiguous().cuda(), c.vt[:, n:n + T].contiguous().cuda())
        n += T
    layer.append(c.kt[:, n:].contiguous().cuda(), c.vt[:, n:].contiguous().cuda())
    ref, tol = c.decode(0, n + 1)
    check(f64(layer.decode(c.query([n + 1])))[0], ref, tol)


def test_equals_the_bf16_prefill_over_the_dequantized_rows():
    """Bit for bit where the scales are powers of two (so the rows are bf16 values), query heads do not
    share query blocks and no item is split over its keys (here: full query blocks, and more of them
    than SMs)."""
    from streaming_kv_cache_duo_gb300 import DuoLayer
    n, T, kinds = 777, 512, [1, 1, 0, 1, 0, 1, 1, 0]
    c = Batch(52, [n + T] * 2, 64, 8, 64, 64, 256, kinds, "int8")
    for name in ("k", "v"):  # the largest of every block is 127 / 64
        t = getattr(c, name + "t").clamp(-127 / 64, 127 / 64)
        t[:, ::BLOCK, :, 0] = 127 / 64
        setattr(c, name + "t", t)
        setattr(c, name, t.double().numpy())
    layer = _layer(c, n + T)
    _fill(c, layer, n)
    plain = DuoLayer(2, 64, 8, 64, 64, 256, n + T, kinds)
    kt, vt = c.kt.clone(), c.vt.clone()
    for x, name in ((kt, "k"), (vt, "v")):
        for b in range(2):
            for h in c.ret:
                rows = c.heads_rows(b, h, n, getattr(c, name))[1]
                x[b, :n, h] = torch.from_numpy(rows.astype(np.float32)).to(torch.bfloat16)
    plain.append(kt[:, :n].contiguous().cuda(), vt[:, :n].contiguous().cuda())
    pick = lambda x: x[:, n:n + T].contiguous().cuda()
    want = plain.prefill(pick(c.qt), pick(c.kt), pick(c.vt))
    assert torch.equal(_run(c, layer, n, T), want)


def test_workspace():
    """The size covers the call, anything may be in it, a smaller one is refused; none is needed
    where no cached row is read."""
    from streaming_kv_cache_duo_gb300 import DuoError, _lib
    n, T = 1300, 20
    c = Batch(55, [n + T], 4, 2, 64, 4, 32, [1, 0], "int8")
    layer = _layer(c, n + T)
    assert _lib.duo_prefill_kv8_workspace_size(layer.handle, 0, T) == 0
    q, k, v = (x[:, :T].contiguous().cuda() for x in (c.qt, c.kt, c.vt))
    first = torch.empty_like(q)
    _lib.duo_attn_prefill_kv8(layer.handle, layer.cache, layer.kv8, q, k, v, T, first, None)
    _fill(c, layer, n)
    need = _lib.duo_prefill_kv8_workspace_size(layer.handle, n, T)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    q, k, v = (x[:, n:].contiguous().cuda() for x in (c.qt, c.kt, c.vt))
    a, b = torch.empty_like(q), torch.empty_like(q)
    _lib.duo_attn_prefill_kv8(layer.handle, layer.cache, layer.kv8, q, k, v, T, a, ws[:need])
    assert bool((ws[need:] == 0xFF).all())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    layer.prefill(q, k, v, out=b, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    _check_chunk(c, n, T, a)
    call = lambda w: _lib.duo_attn_prefill_kv8(layer.handle, layer.cache, layer.kv8, q, k, v, T, a, w)
    for bad in (None, ws[:need - 1]):
        with pytest.raises(DuoError, match="DUO_ERR_WORKSPACE"):
            call(bad)
    with pytest.raises(DuoError, match="DUO_ERR_INVALID_ARG"):
        call(ws[16:])


def test_bad_pages_read_as_nothing_and_are_reported():
    from streaming_kv_cache_duo_gb300 import duo_device_error
    n, T = 400, 50
    c = Batch(53, [n + T], 4, 2, 64, 4, 32, [1, 0], "e4m3")
    layer = _layer(c, n + T, 128)
    _fill(c, layer, n)
    good = layer.block_table.clone()
    pick = lambda x: x[:, n:n + T].contiguous().cuda()
    for bad in (-1, layer.k_codes.shape[0], -(1 << 31)):
        layer.block_table.copy_(good)
        layer.block_table[0, 0, 1] = bad
        out = layer.prefill(pick(c.qt), pick(c.kt), pick(c.vt))
        torch.cuda.synchronize()
        assert duo_device_error() != 0
        assert torch.isfinite(out).all()


def test_refusals():
    from streaming_kv_cache_duo_gb300 import DuoError, _lib
    c = Batch(54, [100], 4, 2, 64, 4, 32, [1, 0], "int8")
    layer = _layer(c, 100)
    q, k, v = (x[:, :10].contiguous().cuda() for x in (c.qt, c.kt, c.vt))
    with pytest.raises(NotImplementedError):
        layer.prefill(q, k, v, kind_mask=2)
    for bad in ((q.float(), k, v), (q, k[:, :9].contiguous(), v), (q, k, v.cpu())):
        with pytest.raises(ValueError):
            layer.prefill(*bad)
    call = lambda kv8, T=10, qq=q: _lib.duo_attn_prefill_kv8(layer.handle, layer.cache, kv8, qq, k, v, T, q, None)
    for args in ((None,), (layer.kv8, 0), (layer.kv8, -1), (layer.kv8, 10, None)):
        with pytest.raises(DuoError, match="DUO_ERR_INVALID_ARG"):
            call(*args)
    layer.cache.n = 101
    with pytest.raises(DuoError, match="DUO_ERR_INVALID_ARG"):
        call(layer.kv8)


@pytest.mark.parametrize("B,T", [(1, 9), (2, 300)], ids=["split", "whole_blocks"])
@pytest.mark.parametrize("which", ["k", "v"])
def test_non_finite_blocks_show_and_stay_with_their_head(B, T, which):
    """An infinity in one cached token of one head: every output of that head's queries is NaN, also
    where its block falls to one of several CTAs; the other heads and sequences are as ever."""
    n = 1500
    c = Batch(57, [n + T] * B, 4, 2, 128, 4, 32, [1, 1], "e4m3")
    layer = _layer(c, n + T)
    bad = {"k": c.kt.clone(), "v": c.vt.clone()}
    bad[which][0, 70, 0] = float("inf")
    layer.append(bad["k"][:, :n].contiguous().cuda(), bad["v"][:, :n].contiguous().cuda())
    got = f64(_run(c, layer, n, T))
    assert np.isnan(got[0, :, :2]).all()
    assert np.isfinite(got[0, :, 2:]).all() and np.isfinite(got[1:]).all()
    clean = _layer(c, n + T)
    clean.append(c.kt[:, :n].contiguous().cuda(), c.vt[:, :n].contiguous().cuda())
    want = f64(_run(c, clean, n, T))
    assert np.array_equal(got[0, :, 2:], want[0, :, 2:]) and np.array_equal(got[1:], want[1:])


def test_captured_chunk_append_and_decode():
    """A chunk's prefill, its append and a decode as one graph, with the workspace that the capture was
    given, replayed on other values than it was captured with: the same bits as the calls one by one."""
    n, T = 900, 70
    c = Batch(58, [n + T] * 2, 8, 2, 128, 4, 64, [1, 0], "int8")
    eager, layer = _layer(c, n + T), _layer(c, n + T)
    cut = lambda x: x[:, n:n + T].contiguous().cuda()
    for x in (eager, layer):
        x.append(c.kt[:, :n].contiguous().cuda(), c.vt[:, :n].contiguous().cuda())
    q, k, v, last = cut(c.qt), cut(c.kt), cut(c.vt), c.query([n + T] * 2)
    qs, ks, vs, ls = (torch.zeros_like(x) for x in (q, k, v, last))
    warm = _layer(c, n + T)  # kernels loaded before the capture
    warm.append(c.kt[:, :n].contiguous().cuda(), c.vt[:, :n].contiguous().cuda())
    warm.prefill(q, k, v)
    warm.append(k, v)
    warm.decode(last)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.prefill(qs, ks, vs)
        layer.append(ks, vs)
        dec = layer.decode(ls)
    for dst, src in ((qs, q), (ks, k), (vs, v), (ls, last)):
        dst.copy_(src)
    graph.replay()
    want = eager.prefill(q, k, v)
    eager.append(k, v)
    want_dec = eager.decode(last)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(dec, want_dec)
    _check_chunk(c, n, T, out, [0, T - 1])


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("T", [9, 300])
def test_blocks_of_scales_far_apart(T, code):
    """Blocks of zeros, of values near the smallest and far above the others, and of one that is all
    that counts: each block's scale is its own."""
    n = 64 * 20 + 17
    c = Batch(59, [n + T] * 2, 4, 2, 128, 4, 32, [1, 1], code)
    kt, vt = c.kt.clone(), c.vt.clone()
    for j in range(20):
        rows = slice(64 * j, 64 * j + 64)
        kt[:, rows] *= [1, 0, 2.0 ** -40, 1.5, 0.3][j % 5]
        vt[:, rows] *= [1, 2.0 ** 3, 0, 2.0 ** -12, 2.0 ** -131, 0.7, 2.0 ** -60][j % 7]
    vt[1, 64 * 3:64 * 4] *= 2.0 ** 60
    for name, t in (("k", kt), ("v", vt)):
        setattr(c, name + "t", t)
        setattr(c, name, t.double().numpy())
    layer = _layer(c, n + T, 128)
    _fill(c, layer, n)
    _check_chunk(c, n, T, _run(c, layer, n, T), [0, T // 2, T - 1])


@pytest.mark.parametrize("Hq,Hkv,kinds", [(8, 8, [1] * 8), (8, 5, None), (8, 4, [1, 0, 1, 1])], ids=["mha", "mixed", "gqa"])
def test_long_chunks_whose_last_parts_differ(Hq, Hkv, kinds):
    """Chunks with about an item per SM, whose keys go on over the SMs without one: parts of one length,
    the last of what is left, from one tile (the first query block) up."""
    n, T = 9000 - 37, 4096 - 5
    if kinds is None:
        Hq, kinds = 10, [1, 1, 1, 1, 0]
    c = Batch(63, [n + T], Hq, Hkv, 64, 64, 256, kinds, "e4m3")
    layer = _layer(c, n + T)
    _fill(c, layer, n)
    out = _run(c, layer, n, T)
    _check_chunk(c, n, T, out, [0, 127, 128, 255, 256, 2000, T - 1])


@pytest.mark.parametrize("layer", ["DuoLayer", "DuoKv8Layer"])
def test_ring_positions_at_the_last_ones_there_are(layer):
    """Streaming heads up to position 2^31 - 5, a chunk whose query block goes on past 2^31: as at small
    positions with the same slots."""
    import streaming_kv_cache_duo_gb300 as duo
    S, R, T, n = 0, 256, 105, (1 << 31) - 110
    rng = np.random.default_rng(64)
    far, near = (getattr(duo, layer)(1, 4, 2, 64, S, R, 1, [0, 0]) for _ in range(2))
    draw = lambda t, h: torch.from_numpy(rng.standard_normal((1, t, h, 64)).astype(np.float32)).bfloat16().cuda()
    k, v = draw(R, 2), draw(R, 2)
    for x, at in ((far, n - R), (near, n % R)):
        x.cache.n = at
        x.append(k, v)
    q, k, v = draw(T, 4), draw(T, 2), draw(T, 2)
    assert far.n == n
    assert torch.equal(far.prefill(q, k, v), near.prefill(q, k, v))
