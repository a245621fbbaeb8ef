"""Appends into 8-bit caches: codes, scales, tails and rings equal the oracle's bit for bit, for
every split of the tokens into calls, and nothing else of the arrays is touched."""

import numpy as np
import pytest
import torch

from kv8_util import BLOCK, expected_rows, f64, normal, ring, scattered_table, slot_of
from oracle.kv8 import quantize_block

pytestmark = pytest.mark.gpu

BUFFERS = ("k_codes", "v_codes", "k_scale", "v_scale", "k_tail", "v_tail", "k_sr", "v_sr", "pos")
CANARY = 77


def _layer(B, Hkv, D, S, R, kinds, cap, code, page=0, rng=None):
    from streaming_kv_cache_duo_gb300 import DuoKv8Layer, DuoKv8PagedLayer
    if page:
        mb = -(-cap // page)
        table, nb = scattered_table(rng, B, sum(kinds), mb)
        return DuoKv8PagedLayer(B, Hkv, Hkv, D, S, R, page, mb, nb, table, kinds, code=code)
    return DuoKv8Layer(B, Hkv, Hkv, D, S, R, cap, kinds, code=code)


def _mark(layer):
    for name in BUFFERS[:-1]:
        t = getattr(layer, name)
        t.view(torch.uint8).fill_(CANARY)


def _block(layer, name, b, r, j):
    """(codes [64, D], scale) of block j of a plane, as float64."""
    codes, scale = getattr(layer, name + "_codes"), getattr(layer, name + "_scale")
    if layer.paged is None:
        return f64(codes[b, r, j * BLOCK:(j + 1) * BLOCK]), scale[b, r, j].item()
    per = layer.block_size // BLOCK
    blk = layer.block_table[b, r, j // per].item()
    return f64(codes[blk, j % per * BLOCK:(j % per + 1) * BLOCK]), scale[blk, j % per].item()


def _check_plane(layer, name, b, r, rows, touched_tail):
    want = expected_rows(rows, layer.code)
    for j, (c, s) in enumerate(zip(want.codes, want.scales)):
        got, gs = _block(layer, name, b, r, j)
        assert np.float32(gs) == s, (name, b, r, j)
        assert np.array_equal(got, c), (name, b, r, j)
    tail = f64(getattr(layer, name + "_tail")[b, r])
    assert np.array_equal(tail[:len(want.tail)], want.tail), (name, b, r)
    raw = getattr(layer, name + "_tail")[b, r].view(torch.uint8).cpu().numpy()
    assert (raw[max(touched_tail, len(want.tail)):] == CANARY).all(), "tail rows past the tokens were written"


def _untouched(layer, name, blocks_written):
    """Codes outside the written blocks keep their canary."""
    codes = getattr(layer, name + "_codes").view(torch.uint8)
    total = codes.numel() // (BLOCK * layer.D)
    marked = (codes.reshape(total, -1) == CANARY).all(1).sum().item()
    assert marked >= total - blocks_written


CASES = [
    # B, Hkv, D, S, R, kinds, calls, page
    (1, 2, 128, 4, 32, [1, 0], [1], 0),
    (2, 3, 64, 4, 32, [1, 0, 1], [63, 1, 1], 0),
    (1, 4, 128, 64, 256, [0, 1, 1, 0], [64, 65, 127, 1, 300], 0),
    (3, 2, 128, 0, 5, [1, 0], [200, 57, 3, 500], 128),
    (2, 2, 64, 3, 20, [1, 1], [130, 62, 1, 255, 7], 256),
    (1, 2, 128, 4, 32, [0, 0], [100, 7], 0),
    (1, 2, 64, 4, 32, [1, 0], [5000], 384),
]


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("case", CASES, ids=[f"case{i}" for i in range(len(CASES))])
def test_uniform_appends_match_the_oracle(case, code):
    from streaming_kv_cache_duo_gb300 import duo_device_error
    B, Hkv, D, S, R, kinds, calls, page = case
    rng = np.random.default_rng(5)
    n = sum(calls)
    kt, k = normal(rng, B, n, Hkv, D)
    vt, v = normal(rng, B, n, Hkv, D, scale=3.0)
    layer = _layer(B, Hkv, D, S, R, kinds, n + 70, code, page, rng)
    _mark(layer)
    at, touched = 0, 0
    for T in calls:
        layer.append(kt[:, at:at + T].contiguous().cuda(), vt[:, at:at + T].contiguous().cuda())
        at += T
        touched = max(touched, at % BLOCK)
    assert duo_device_error() == 0 and layer.n == n
    ret = [h for h in range(Hkv) if kinds[h]]
    stream = [h for h in range(Hkv) if not kinds[h]]
    for b in range(B):
        for name, x in (("k", k), ("v", v)):
            for r, h in enumerate(ret):
                _check_plane(layer, name, b, r, x[b, :, h], BLOCK)
            for s, h in enumerate(stream):
                pos, rows = ring(x[b, :, h], S, R)
                got = f64(getattr(layer, name + "_sr")[b, s])
                assert np.array_equal(got[pos >= 0], rows[pos >= 0])
                if s == 0:
                    assert np.array_equal(layer.pos[b].cpu().numpy(), pos)
    if ret:
        for name in ("k", "v"):
            _untouched(layer, name, B * len(ret) * (n // BLOCK))


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_single_tokens_leave_the_same_cache_as_one_call(code):
    B, Hkv, D, S, R, n = 2, 2, 128, 4, 32, 3 * BLOCK + 11
    rng = np.random.default_rng(6)
    kt, _ = normal(rng, B, n, Hkv, D)
    vt, _ = normal(rng, B, n, Hkv, D)
    one = _layer(B, Hkv, D, S, R, [1, 0], n, code)
    one.append(kt.cuda(), vt.cuda())
    many = _layer(B, Hkv, D, S, R, [1, 0], n, code)
    for t in range(n):
        many.append(kt[:, t:t + 1].contiguous().cuda(), vt[:, t:t + 1].contiguous().cuda())
    for name in BUFFERS:
        a, b = getattr(one, name).view(torch.uint8), getattr(many, name).view(torch.uint8)
        if "tail" in name:  # rows of the open block (earlier blocks passed through single tokens' tails)
            a, b = a[:, :, :n % BLOCK], b[:, :, :n % BLOCK]
        assert torch.equal(a, b), name


@pytest.mark.parametrize("D,code,lead", [(64, "int8", 0), (128, "e4m3", 64), (64, "e4m3", 37), (128, "int8", 101)])
def test_long_calls_leave_the_same_cache_as_short_ones(D, code, lead):
    """Calls with more chunks than fit on the GPU at once, from a block's start and from inside one."""
    B, Hkv, S, R, n = 2, 9, 70, 300, 9000 + 17
    kinds = [1, 1, 0, 1, 1, 1, 1, 1, 1]
    rng = np.random.default_rng(60)
    kt, vt = (normal(rng, B, lead + n, Hkv, D)[0].cuda() for _ in range(2))
    cut = lambda x, a, b: x[:, a:b].contiguous()
    one, many = (_layer(B, Hkv, D, S, R, kinds, lead + n, code) for _ in range(2))
    for layer in (one, many):
        _mark(layer)
        if lead:
            layer.append(cut(kt, 0, lead), cut(vt, 0, lead))
    one.append(cut(kt, lead, lead + n), cut(vt, lead, lead + n))
    for t in range(lead, lead + n, 1000):
        many.append(cut(kt, t, min(t + 1000, lead + n)), cut(vt, t, min(t + 1000, lead + n)))
    open_rows = (lead + n) % BLOCK
    for name in BUFFERS:
        a, b = getattr(one, name).view(torch.uint8), getattr(many, name).view(torch.uint8)
        if "tail" in name:
            a, b = a[:, :, :open_rows], b[:, :, :open_rows]
        assert torch.equal(a, b), name


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_long_ragged_calls_leave_the_same_cache_as_short_ones(code):
    """A packed batch of many sequences (none, one or thousands of new tokens, from anywhere in a
    block, skipped ones between) in one call, and sequence by sequence."""
    from streaming_kv_cache_duo_gb300 import duo_device_error
    B, Hkv, D, S, R, page = 40, 9, 64, 4, 32, 128
    kinds = [1, 1, 1, 1, 0, 1, 1, 1, 1]
    rng = np.random.default_rng(61)
    start = [int(x) for x in rng.integers(0, 200, B)]
    new = [int(x) for x in rng.choice([0, 1, 5, 63, 64, 65, 300, 700], B)]
    new[3], new[20] = 3000, 2049
    skip = (5, 21)
    cap = max(s + t for s, t in zip(start, new))
    mb = -(-cap // page)
    table, _ = scattered_table(rng, B, 8, mb)
    from streaming_kv_cache_duo_gb300 import DuoKv8PagedLayer
    nb = int(table.max()) + 1
    layers = [DuoKv8PagedLayer(B, Hkv, Hkv, D, S, R, page, mb, nb, table, kinds, code=code) for _ in range(2)]
    total = sum(new)
    assert total > 8700
    kt, vt = (torch.from_numpy(rng.standard_normal((sum(start) + total, Hkv, D)).astype(np.float32)).bfloat16().cuda()
              for _ in range(2))
    first = sum(start)
    for layer in layers:
        _mark(layer)
        layer.append_ragged(kt[:first].contiguous(), vt[:first].contiguous(), _maps(table, page, [0] * B, start))
    layers[0].append_ragged(kt[first:].contiguous(), vt[first:].contiguous(), _maps(table, page, start, new, skip=skip))
    at = first
    for b in range(B):
        if new[b] and b not in skip:
            alone = [new[b] if i == b else 0 for i in range(B)]
            layers[1].append_ragged(kt[at:at + new[b]].contiguous(), vt[at:at + new[b]].contiguous(),
                                    _maps(table, page, start, alone))
        at += new[b]
    torch.cuda.synchronize()
    assert duo_device_error() == 0
    held = [s + (0 if b in skip else t) for b, (s, t) in enumerate(zip(start, new))]
    for name in BUFFERS:
        a, b = (getattr(x, name).view(torch.uint8) for x in layers)
        if "tail" in name:
            for i, n in enumerate(held):
                assert torch.equal(a[i, :, :n % BLOCK], b[i, :, :n % BLOCK]), (name, i)
        else:
            assert torch.equal(a, b), name


def _edge_block(kind, D, rng):
    """64 rows [64, D] of bf16 values where the rounding can go wrong."""
    x = rng.standard_normal((BLOCK, D))
    if kind == "zeros":
        x[:] = 0
    elif kind == "one_outlier":
        x[17, D - 1] = -3e38
    elif kind == "subnormal":
        x = x * 1e-40
    elif kind == "tiny_scale":
        x = np.sign(x) * 2.0 ** -126
    elif kind == "ties":  # quotients on half steps: scale is exactly 1 (int8) or 2^-n (e4m3)
        x = rng.integers(-254, 255, (BLOCK, D)) / 2.0
        x[0, 0] = 127.0
    elif kind == "powers":
        x = np.sign(x) * np.exp2(rng.integers(-20, 9, (BLOCK, D)))
    elif kind in ("inf", "-inf", "nan"):
        x[63, 5] = float(kind)
    return x


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_edge_blocks_match_the_oracle(code, D):
    kinds = ["zeros", "one_outlier", "subnormal", "tiny_scale", "ties", "powers", "inf", "-inf", "nan"]
    rng = np.random.default_rng(7)
    x = torch.from_numpy(np.concatenate([_edge_block(s, D, rng) for s in kinds]).astype(np.float32)).to(torch.bfloat16)
    layer = _layer(1, 1, D, 0, 1, [1], len(x), code)
    layer.append(x[None, :, None].contiguous().cuda(), x[None, :, None].contiguous().cuda())
    vals = x.double().numpy()
    for j, kind in enumerate(kinds):
        c, s = quantize_block(vals[j * BLOCK:(j + 1) * BLOCK], code)
        got, gs = _block(layer, "k", 0, 0, j)
        assert np.array_equal(got, c), kind
        assert (np.isnan(gs) and np.isnan(s)) or np.float32(gs) == s, kind


def _maps(table, page, start, new, pad=0, skip=()):
    """The slot map of new[b] tokens from start[b] on (sequences in `skip` not stored)."""
    from streaming_kv_cache_duo_gb300 import DuoSlotMap
    B, planes = table.shape[:2]
    t = table.cpu().numpy()
    seq, pos, slots = [], [], []
    for b in range(B):
        for i in range(new[b]):
            p = start[b] + i
            seq.append(b)
            pos.append(-1 if b in skip else p)
            slots.append([-1 if b in skip else int(t[b, r, p // page]) * page + p % page for r in range(planes)])
    seq += [-1] * pad
    pos += [-1] * pad
    slots += [[-1] * planes] * pad
    dev = lambda x, d: torch.tensor(x, dtype=d, device="cuda")
    return DuoSlotMap(dev(np.cumsum([0] + list(new)), torch.int32), dev(seq, torch.int32), dev(pos, torch.int32),
                      dev(np.array(slots, np.int64).reshape(-1, planes), torch.int64))


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("D,page", [(128, 128), (64, 256)])
def test_ragged_steps_match_the_oracle(code, D, page):
    from streaming_kv_cache_duo_gb300 import duo_device_error
    B, Hkv, S, R, kinds = 5, 3, 4, 32, [1, 0, 1]
    rng = np.random.default_rng(8)
    # tokens per call and sequence: none, one, block ends from inside a block and from its
    # start, several blocks that end in the middle of one
    calls = [[1, 64, 63, 0, 200], [63, 1, 2, 1, 130], [0, 190, 63, 62, 1], [65, 3, 64, 1, 0], [1, 1, 1, 1, 1]]
    L = np.sum(calls, 0)
    cap = int(L.max()) + 5
    kt, k = normal(rng, B, cap, Hkv, D)
    vt, v = normal(rng, B, cap, Hkv, D)
    layer = _layer(B, Hkv, D, S, R, kinds, cap, code, page, rng)
    _mark(layer)
    start = [0] * B
    for ci, new in enumerate(calls):
        pad = [0, 3, 0, 70, 1][ci]
        pick = lambda x: torch.cat([x[b, start[b]:start[b] + new[b]] for b in range(B)] + [x[0, :pad]]).contiguous().cuda()
        layer.append_ragged(pick(kt), pick(vt), _maps(layer.block_table, page, start, new, pad))
        start = [s + t for s, t in zip(start, new)]
    assert duo_device_error() == 0
    for b in range(B):
        for name, x in (("k", k), ("v", v)):
            for r, h in enumerate([0, 2]):
                _check_plane(layer, name, b, r, x[b, :L[b], h], BLOCK)
            pos, rows = ring(x[b, :L[b], 1], S, R)
            assert np.array_equal(f64(getattr(layer, name + "_sr")[b, 0])[pos >= 0], rows[pos >= 0])
            assert np.array_equal(layer.pos[b].cpu().numpy(), pos)


def test_skipped_sequences_and_empty_batches_change_nothing():
    from streaming_kv_cache_duo_gb300 import duo_device_error
    B, Hkv, D, page = 3, 2, 64, 128
    rng = np.random.default_rng(9)
    kt, _ = normal(rng, B, 200, Hkv, D)
    layer = _layer(B, Hkv, D, 4, 32, [1, 0], 300, "int8", page, rng)
    _mark(layer)
    before = {name: getattr(layer, name).clone() for name in BUFFERS}
    layer.append_ragged(kt[0, :0].contiguous().cuda(), kt[0, :0].contiguous().cuda(),
                        _maps(layer.block_table, page, [0] * B, [0] * B))
    new = [100, 64, 7]
    x = torch.cat([kt[b, :new[b]] for b in range(B)]).contiguous().cuda()
    layer.append_ragged(x, x, _maps(layer.block_table, page, [0] * B, new, skip=(0, 2)))
    assert duo_device_error() == 0
    for name in ("k_tail", "v_tail", "k_sr", "v_sr", "pos"):
        for b in (0, 2):
            a = getattr(layer, name)[b].contiguous().view(torch.uint8)
            assert torch.equal(a, before[name][b].contiguous().view(torch.uint8)), name
    _check_plane(layer, "k", 1, 0, kt[1, :64, 0].double().numpy(), 0)
    _untouched(layer, "k", 1)


def test_bad_slots_and_sequences_are_reported_and_skipped():
    from streaming_kv_cache_duo_gb300 import _lib
    B, Hkv, D, page = 2, 1, 64, 128
    rng = np.random.default_rng(10)
    kt, k = normal(rng, B, 64, Hkv, D)
    for bad in ("slot_high", "slot_low", "slot_odd", "seq_high", "cu"):
        layer = _layer(B, Hkv, D, 0, 4, [1], 300, "int8", page, rng)
        _mark(layer)
        m = _maps(layer.block_table, page, [0, 0], [64, 64])
        if bad == "slot_high":
            m.slots[63, 0] = layer.k_codes.shape[0] * page + 63
        elif bad == "slot_low":
            m.slots[63, 0] = 5
        elif bad == "slot_odd":
            m.slots[63, 0] += 1
        elif bad == "seq_high":
            m.token_seq[:64] = B
        else:
            m.cu_new[1] = 200
        x = torch.cat([kt[0], kt[1]]).contiguous().cuda()
        layer.append_ragged(x, x, m)
        torch.cuda.synchronize()
        assert _lib.duo_device_error() != 0, bad
        if bad != "cu":
            _check_plane(layer, "k", 1, 0, k[1, :, 0], 0)
            _untouched(layer, "k", 1)
        assert _lib.duo_device_error() == 0
    # a table entry that is no block, in a uniform append
    layer = _layer(B, Hkv, D, 0, 4, [1], 300, "int8", page, rng)
    _mark(layer)
    layer.block_table[0, 0, 0] = layer.k_codes.shape[0]
    layer.append(kt.cuda(), kt.cuda())
    torch.cuda.synchronize()
    assert _lib.duo_device_error() != 0
    _check_plane(layer, "k", 1, 0, k[1, :, 0], 0)
    _untouched(layer, "k", 1)


def test_refusals():
    from streaming_kv_cache_duo_gb300 import DuoError, DuoKv8Layer, _lib
    layer = _layer(2, 2, 64, 4, 32, [1, 0], 100, "int8")
    x = torch.zeros(2, 101, 2, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(DuoError, match="DUO_ERR_CAPACITY"):
        layer.append(x, x)
    assert layer.n == 0
    for bad in (x[:1, :1], x[:, :1].float(), x[:, :1].cpu(), x[:, :4, :, :32]):
        with pytest.raises(ValueError):
            layer.append(bad, bad)
    with pytest.raises(ValueError):
        DuoKv8Layer(1, 2, 2, 64, 4, 32, 100, [1, 0], code="fp4")
    one = x[:, :1].contiguous()
    call = lambda kv8, a=one, b=one: _lib.duo_kv_append_kv8(layer.handle, layer.cache, kv8, a, b, 1)
    with pytest.raises(DuoError, match="DUO_ERR_INVALID_ARG"):
        call(None)
    with pytest.raises(DuoError, match="DUO_ERR_INVALID_ARG"):
        call(layer.kv8, None)
    for field, value in (("code_type", 2), ("code_type", -1), ("k_codes", None), ("v_scale", None), ("k_tail", 0),
                         ("v_codes", layer.kv8.v_codes + 8)):
        kv8 = _lib.duo_kv8_cache(*[getattr(layer.kv8, f) for f, _ in _lib.duo_kv8_cache._fields_])
        setattr(kv8, field, value)
        with pytest.raises(DuoError, match="DUO_ERR_INVALID_ARG"):
            call(kv8)
    stream_pool = _lib.duo_paged(layer.pos.data_ptr(), 128, 1, 4, layer.pos.data_ptr())
    with pytest.raises(DuoError, match="DUO_ERR_UNSUPPORTED"):
        _lib.duo_kv_append_kv8_paged(layer.handle, layer.cache, stream_pool, layer.kv8, one, one, 1)
    for size in (64, 100, 0):
        with pytest.raises(DuoError, match="DUO_ERR_UNSUPPORTED"):
            _lib.duo_kv_append_kv8_paged(layer.handle, layer.cache, _lib.duo_paged(layer.pos.data_ptr(), size, 1, 4, None),
                                         layer.kv8, one, one, 1)
    with pytest.raises(DuoError, match="DUO_ERR_UNSUPPORTED"):  # 2^31 rows of codes
        _lib.duo_kv_append_kv8_paged(layer.handle, layer.cache,
                                     _lib.duo_paged(layer.pos.data_ptr(), 128, 1, 1 << 24, None), layer.kv8, one, one, 1)
    with pytest.raises(DuoError, match="DUO_ERR_INVALID_ARG"):
        _lib.duo_kv_append_kv8_ragged(layer.handle, layer.cache, _lib.duo_paged(layer.pos.data_ptr(), 128, 1, 4, None),
                                      layer.kv8, None, 2, one, one)
    assert layer.n == 0
