"""Decode over 8-bit caches against attention in 64 bits over the rows the cache stands for, each
output within a bound derived from the roundings of the kernel (kv8_util.attend)."""

import numpy as np
import pytest
import torch

from kv8_util import BLOCK, Batch, check, f64, scattered_table

pytestmark = pytest.mark.gpu


def _layer(c, cap, page=0, rng=None, kinds=None):
    from streaming_kv_cache_duo_gb300 import DuoKv8Layer, DuoKv8PagedLayer
    if page:
        mb = -(-cap // page)
        table, nb = scattered_table(rng, c.B, len(c.ret), mb)
        return DuoKv8PagedLayer(c.B, c.Hq, c.Hkv, c.D, c.S, c.R, page, mb, nb, table, c.kinds, code=c.code)
    return DuoKv8Layer(c.B, c.Hq, c.Hkv, c.D, c.S, c.R, cap, c.kinds, code=c.code)


def _poison(layer, n):
    """NaN in everything a decode at n tokens must not use: open-block rows past the tokens,
    blocks past the last full one, empty ring slots."""
    full = n // BLOCK
    for name in ("k", "v"):
        getattr(layer, name + "_tail")[:, :, n % BLOCK:] = float("nan")
        if n < layer.S + layer.R:
            getattr(layer, name + "_sr")[:, :, n:] = float("nan")
        if layer.paged is None:
            getattr(layer, name + "_scale")[:, :, full:] = float("nan")
            if layer.code == "e4m3":
                getattr(layer, name + "_codes").view(torch.uint8)[:, :, full * BLOCK:] = 0x7F


def _check(layer, c, n, out):
    from streaming_kv_cache_duo_gb300 import duo_device_error
    torch.cuda.synchronize()
    assert duo_device_error() == 0
    got = f64(out)
    for b in range(c.B):
        ref, tol = c.decode(b, n)
        check(got[b], ref, tol, f"sequence {b} at {n} tokens")


SHAPES = [
    # B, Hq, Hkv, D, S, R, kinds
    (1, 4, 4, 128, 4, 32, [1, 0, 1, 0]),
    (2, 4, 2, 64, 4, 32, [1, 0]),
    (1, 8, 2, 128, 64, 256, [0, 1]),
    (1, 16, 2, 64, 0, 5, [1, 1]),
    (2, 8, 1, 128, 3, 20, [1]),
    (1, 8, 2, 64, 130, 190, [0, 0]),
]
LENS = [1, 2, 63, 64, 65, 127, 128, 255, 256, 257, 319, 320, 1023, 1111, 2500]


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("shape", SHAPES, ids=[f"shape{i}" for i in range(len(SHAPES))])
def test_lengths(shape, code):
    B, Hq, Hkv, D, S, R, kinds = shape
    c = Batch(30, [max(LENS)] * B, Hq, Hkv, D, S, R, kinds, code)
    layer = _layer(c, max(LENS))
    at = 0
    for n in LENS:
        layer.append(c.kt[:, at:n].contiguous().cuda(), c.vt[:, at:n].contiguous().cuda())
        at = n
        keep = {k: getattr(layer, k).clone() for k in ("k_tail", "v_tail", "k_sr", "v_sr", "k_scale", "v_scale")}
        _poison(layer, n)
        out = layer.decode(c.query([n] * B))
        _check(layer, c, n, out)
        for k, t in keep.items():
            getattr(layer, k).copy_(t)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("page,D", [(128, 128), (256, 64), (384, 128)])
def test_paged_equals_contiguous_bit_for_bit(page, D, code):
    n = 1999
    c = Batch(31, [n, n], 8, 2, D, 4, 32, [1, 0], code)
    flat = _layer(c, n)
    paged = _layer(c, n, page, np.random.default_rng(1))
    c.fill(flat)
    c.fill(paged, 700)
    q = c.query([n, n])
    a, b = flat.decode(q), paged.decode(q)
    assert torch.equal(a, b)
    _check(flat, c, n, a)
    lens = torch.full((2,), n, dtype=torch.int32, device="cuda")
    assert torch.equal(flat.decode_varlen(q, lens, n), a)
    assert torch.equal(paged.decode_varlen(q, lens, n), a)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("B,Hq,Hkv,D,kinds,most", [
    (7, 8, 2, 128, [1, 0], 1500),      # fewer tiles than SMs, every unit short or split
    (40, 16, 4, 64, [1, 0, 1, 0], 900),  # more units than SMs
    (3, 2, 2, 128, [1, 1], 6000),
    (300, 2, 1, 64, [1], 130),         # more sequences than a CTA has threads
])
def test_ragged_lengths_on_the_device(B, Hq, Hkv, D, kinds, most, code):
    rng = np.random.default_rng(32)
    lens = rng.integers(0, most + 1, B)
    lens[:4] = [most, 0, 64, 1][:min(4, B)]
    c = Batch(33, lens, Hq, Hkv, D, 4, 32, kinds, code)
    layer = _ragged_layer(c, lens, 128, rng)
    out = layer.decode_varlen(c.query(lens), torch.from_numpy(lens.astype(np.int32)).cuda(), most + 7)
    from streaming_kv_cache_duo_gb300 import duo_device_error
    torch.cuda.synchronize()
    assert duo_device_error() == 0
    got = f64(out)
    for b in range(B) if B <= 40 else list(range(0, B, 17)):
        ref, tol = c.decode(b, int(lens[b]))
        check(got[b], ref, tol, f"sequence {b} of {lens[b]} tokens")
    empty = [b for b in range(B) if lens[b] == 0]
    assert not np.any(got[empty])


def _ragged_layer(c, lens, page, rng):
    """A paged layer of the batch's sequences, appended through the device's tables."""
    from streaming_kv_cache_duo_gb300 import DuoBlockPool, DuoKv8PagedLayer
    mb = -(-(max(max(lens), 1) + 8) // page)
    nb = c.B * len(c.ret) * mb + 2
    N = int(sum(lens)) + 5
    pool = DuoBlockPool(c.B, len(c.ret), page, mb, nb, N)
    pool.free_list.copy_(torch.from_numpy(rng.permutation(nb).astype(np.int32)))
    layer = DuoKv8PagedLayer(c.B, c.Hq, c.Hkv, c.D, c.S, c.R, page, mb, nb, pool.block_table, c.kinds, code=c.code)
    m = pool.update(torch.from_numpy(np.asarray(lens).astype(np.int32)).cuda())
    k, v = c.packed([0] * c.B, lens)
    pad = torch.full((5,) + tuple(k.shape[1:]), float("nan"), dtype=torch.bfloat16, device="cuda")
    layer.append_ragged(torch.cat([k, pad]), torch.cat([v, pad]), m)
    return layer


def test_lengths_are_clamped_to_the_plan():
    c = Batch(34, [500], 4, 2, 64, 4, 32, [1, 0], "int8")
    layer = _layer(c, 500)
    c.fill(layer)
    q = c.query([256])
    a = layer.decode_varlen(q, torch.tensor([9999], dtype=torch.int32, device="cuda"), 256)
    b = layer.decode_varlen(q, torch.tensor([-5], dtype=torch.int32, device="cuda"), 256)
    ref, tol = c.decode(0, 256)
    # (ring slots hold the 500-token state: only the retrieval heads stand for 256 tokens, four full blocks)
    check(f64(a)[0, :2], ref[:2], tol[:2])
    assert not f64(b).any()


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("q_scale,k_scale", [(2.0 ** 100, 2.0 ** -100), (2.0 ** -60, 2.0 ** 60), (8.0, 1.0), (1e-30, 1.0)])
def test_ranges_far_from_one(q_scale, k_scale, code):
    """q and k of any size: neither passes through fp16 unscaled. q_scale 8: peaked rows."""
    n = 700
    c = Batch(35, [n], 8, 2, 128, 4, 32, [1, 0], code, scale=k_scale)
    c.qt = (c.qt.double() * q_scale).to(torch.bfloat16)
    c.q = c.qt.double().numpy()
    c.vt = (c.vt.double() * 2.0 ** 90).to(torch.bfloat16)
    c.v = c.vt.double().numpy()
    layer = _layer(c, n)
    c.fill(layer)
    _check(layer, c, n, layer.decode(c.query([n])))


def test_a_dominant_key_late_and_many_small_ones():
    """The running maximum jumps by far more than the lazy limit late in the row; and 20000 keys
    at 2^-14 of one key's weight still count for what they weigh."""
    n, D = 20000, 64
    c = Batch(36, [n], 2, 1, D, 4, 32, [1], "int8")
    c.k[:] = 0
    c.q[:] = 0
    c.q[..., 0] = 8.0
    c.k[..., 0] = -1.0
    c.k[0, 17777, 0, 0] = 8.75  # 9.75 * 8 / 8 = 9.75 nats above the others: 2^-14.07 each
    c.v[:] = 1.0
    c.v[0, 17777] = -1.0
    for name in ("q", "k", "v"):
        setattr(c, name + "t", torch.from_numpy(getattr(c, name)).to(torch.bfloat16))
        assert np.array_equal(getattr(c, name + "t").double().numpy(), getattr(c, name))
    layer = _layer(c, n)
    c.fill(layer)
    out = layer.decode(c.query([n]))
    ref, _ = c.decode(0, n)
    assert -0.2 < ref[0, 0] < 0.2  # the two sides nearly cancel
    _check(layer, c, n, out)


def test_non_finite_blocks_show_and_stay_with_their_head():
    n = 300
    c = Batch(37, [n], 4, 2, 64, 4, 32, [1, 1], "int8")
    kt = c.kt.clone()
    kt[0, 70, 0, 3] = float("inf")
    layer = _layer(c, n)
    layer.append(kt.cuda(), c.vt.cuda())
    got = f64(layer.decode(c.query([n])))
    assert np.isnan(got[0, :2]).all()
    ref, tol = c.decode(0, n)
    check(got[0, 2:], ref[2:], tol[2:])


@pytest.mark.parametrize("which", ["k", "v"])
def test_a_non_finite_block_among_many_ctas(which):
    """The same where the head is shared by many CTAs, of which one has the block."""
    n = 70000
    c = Batch(42, [n], 4, 2, 64, 4, 32, [1, 1], "e4m3")
    bad = {"k": c.kt.clone(), "v": c.vt.clone()}
    bad[which][0, 40000, 0] = float("nan")
    layer, clean = _layer(c, n), _layer(c, n)
    layer.append(bad["k"].cuda(), bad["v"].cuda())
    c.fill(clean)
    got, want = f64(layer.decode(c.query([n]))), f64(clean.decode(c.query([n])))
    assert np.isnan(got[0, :2]).all()
    assert np.array_equal(got[0, 2:], want[0, 2:])


def test_bad_blocks_are_reported_and_skipped():
    from streaming_kv_cache_duo_gb300 import duo_device_error
    n, page = 600, 128
    c = Batch(38, [n], 4, 2, 64, 4, 32, [1, 0], "int8")
    layer = _layer(c, n, page, np.random.default_rng(2))
    c.fill(layer)
    good = layer.block_table.clone()
    for bad in (-1, layer.k_codes.shape[0], 0x7fffffff, -(1 << 31)):
        layer.block_table.copy_(good)
        layer.block_table[0, 0, 1] = bad
        out = f64(layer.decode(c.query([n])))
        torch.cuda.synchronize()
        assert duo_device_error() != 0
        assert np.isfinite(out).all()
        ref, tol = c.decode(0, n)
        check(out[0, 2:], ref[2:], tol[2:])  # the streaming head
    # entries past the tokens may hold anything
    layer.block_table.copy_(good)
    layer.cache.n = 256
    layer.block_table[0, 0, 2:] = -1
    layer.decode(c.query([256]))
    torch.cuda.synchronize()
    assert duo_device_error() == 0


def test_workspace_content_and_streams():
    """Dirty workspaces give the same bits; so do two layers decoding at once on two streams."""
    n = 5000
    c = Batch(39, [n], 8, 2, 128, 4, 32, [1, 0], "e4m3")
    a, b = _layer(c, n), _layer(c, n)
    c.fill(a)
    c.fill(b)
    q = c.query([n])
    first = a.decode(q)
    a.workspace.fill_(0xFF)
    assert torch.equal(a.decode(q), first)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.empty_like(q) for _ in range(2)]
    for _ in range(20):
        for layer, s, o in zip((a, b), streams, outs):
            layer.decode(q, out=o, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], first) and torch.equal(outs[1], first)
    _check(a, c, n, first)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_a_serving_run_captured_and_replayed(code):
    """Tables, ragged append and decode of a batch as one CUDA graph: sequences grow by their own
    numbers of tokens, one finishes and its place is taken by a new one, the pool runs out once."""
    from streaming_kv_cache_duo_gb300 import DuoBlockPool, DuoKv8PagedLayer, _lib
    B, Hq, Hkv, D, S, R, page, N = 4, 4, 2, 64, 4, 32, 128, 200
    kinds = [1, 0]
    rng = np.random.default_rng(40)
    room = 500
    c = Batch(41, [room] * B, Hq, Hkv, D, S, R, kinds, code)
    mb, nb = 5, 8
    pool = DuoBlockPool(B, 1, page, mb, nb, N)
    layer = DuoKv8PagedLayer(B, Hq, Hkv, D, S, R, page, mb, nb, pool.block_table, kinds, code=code)
    new = torch.zeros(B, dtype=torch.int32, device="cuda")
    k = torch.zeros(N, Hkv, D, dtype=torch.bfloat16, device="cuda")
    v, q = torch.zeros_like(k), torch.zeros(B, Hq, D, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    layer.decode_varlen(q, pool.seq_lens, mb * page, out=out)  # (first launches before the capture)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m = pool.update(new)
        layer.append_ragged(k, v, m)
        layer.decode_varlen(q, pool.seq_lens, mb * page, out=out)
    at = [0] * B
    steps = [[70, 1, 64, 0], [1, 63, 65, 1], [60, 64, 1, 3], [1, 1, -1, 127], [129, 1, 5, 1], [1, 1, 30, 1],
             [1, 130, 1, 1], [30, 1, 1, 1]]
    turned_down = 0
    for new_lens in steps:
        packed, qs, want, took = [], [], [], list(at)
        free = nb - sum(-(-x // page) for x in at) + sum(-(-at[b] // page) for b in range(B) if new_lens[b] < 0)
        starved = False
        for b in range(B):
            t = new_lens[b]
            if t < 0:
                took[b] = 0
                continue
            packed += [(b, at[b] + i) for i in range(t)]
            need = -(-(at[b] + t) // page) - -(-at[b] // page)
            if need and (starved or need > free):
                starved = True
                turned_down += 1
                continue
            free -= need
            took[b] = at[b] + t
        new.copy_(torch.tensor(new_lens, dtype=torch.int32))
        idx = torch.tensor(packed).T
        k.fill_(float("nan"))
        v.fill_(float("nan"))
        k[:len(packed)] = c.kt[idx[0], idx[1]].cuda()
        v[:len(packed)] = c.vt[idx[0], idx[1]].cuda()
        q.copy_(c.query(took))
        g.replay()
        torch.cuda.synchronize()
        assert pool.seq_lens.tolist() == took
        assert (_lib.duo_device_error() != 0) == starved
        got = f64(out)
        for b in range(B):
            ref, tol = c.decode(b, took[b])
            check(got[b], ref, tol, f"sequence {b} of {took[b]} tokens")
        at = took
    assert turned_down


def test_refusals():
    from streaming_kv_cache_duo_gb300 import DuoError, _lib
    c = Batch(42, [10], 4, 2, 64, 4, 32, [1, 0], "int8")
    layer = _layer(c, 100)
    q = c.query([10])
    with pytest.raises(DuoError, match="DUO_ERR_INVALID_ARG"):
        layer.decode(q)  # nothing appended yet
    c.fill(layer)
    lens = torch.tensor([10], dtype=torch.int32, device="cuda")
    for max_len in (0, -1, 101, 1 << 31):
        with pytest.raises(DuoError, match="DUO_ERR_INVALID_ARG"):
            layer.decode_varlen(q, lens, max_len)
    for bad in (q.float(), q.cpu(), q[:, :2], q.transpose(1, 2)):
        with pytest.raises(ValueError):
            layer.decode(bad)
    with pytest.raises(ValueError):
        layer.decode_varlen(q, lens.long(), 10)
    with pytest.raises(DuoError, match="DUO_ERR_WORKSPACE"):
        _lib.duo_attn_decode_kv8(layer.handle, layer.cache, layer.kv8, q, q, layer.workspace[:256])
    with pytest.raises(DuoError, match="DUO_ERR_WORKSPACE"):
        _lib.duo_attn_decode_kv8(layer.handle, layer.cache, layer.kv8, q, q, None)
    with pytest.raises(DuoError, match="DUO_ERR_INVALID_ARG"):
        _lib.duo_attn_decode_kv8(layer.handle, layer.cache, layer.kv8, q, q, layer.workspace[16:])
    with pytest.raises(DuoError, match="DUO_ERR_INVALID_ARG"):
        _lib.duo_attn_decode_kv8(layer.handle, layer.cache, None, q, q, layer.workspace)
    with pytest.raises(NotImplementedError):
        layer.append_varlen(None, None, None)
