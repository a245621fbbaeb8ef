"""Packed chunks and single tokens over bf16 paged caches against softmax attention in 64 bits. Rows that
take no part (blocks not written, padding, other sequences' ends) hold NaN throughout."""

import ctypes

import numpy as np
import pytest
import torch

from kv8_util import attend, check
from ragged_util import f64, kinds_of, normal, scattered_table, slot_map

pytestmark = pytest.mark.gpu
NAN = float("nan")


class Batch:
    """Sequences of (cached, new) tokens: values per position, and a paged layer that holds the cached ones."""

    def __init__(self, seed, seqs, Hq, Hkv, n_ret, D, S, R, page, appended=False, scale=1.0):
        from streaming_kv_cache_duo_gb300 import DuoPagedLayer
        rng = np.random.default_rng(seed)
        self.rng, self.seqs, self.B, self.g = rng, seqs, len(seqs), Hq // Hkv
        self.Hq, self.Hkv, self.D, self.S, self.R, self.page = Hq, Hkv, D, S, R, page
        self.kinds = kinds_of(Hkv, n_ret)
        self.k, self.v, self.q = [], [], []
        for n, T in seqs:
            self.k.append(normal(rng, n + T, Hkv, D, scale=scale))
            self.v.append(normal(rng, n + T, Hkv, D))
            self.q.append(normal(rng, n + T, Hq, D, scale=scale))
        mb = -(-max(max(n + T for n, T in seqs), 1) // page)
        self.table, nb = scattered_table(rng, self.B, max(1, n_ret), mb)
        self.layer = DuoPagedLayer(self.B, Hq, Hkv, D, S, R, page, mb, nb, self.table if n_ret else None, self.kinds)
        for name in ("k_full", "v_full", "k_sr", "v_sr"):
            getattr(self.layer, name).fill_(NAN)
        self.append([0] * self.B, [n for n, _ in seqs])
        if appended:
            self.append([n for n, _ in seqs], [T for _, T in seqs])

    def map(self, start, new, pad=0):
        return slot_map(self.table if sum(self.kinds) else None, self.page, start, new, pad)

    def packed(self, x, start, new, pad=0):
        rows = [x[b][0][s or 0:(s or 0) + t] for b, (s, t) in enumerate(zip(start, new))]
        if pad:
            rows.append(torch.full((pad,) + tuple(x[0][0].shape[1:]), NAN, dtype=torch.bfloat16))
        return torch.cat(rows).cuda()

    def append(self, start, new):
        if sum(new):
            self.layer.append_ragged(self.packed(self.k, start, new), self.packed(self.v, start, new), self.map(start, new))

    def expected(self, b, i, j):
        """Output and bound of sequence b's query at position i, query head j."""
        h = j // self.g
        at = np.arange(i + 1)
        see = np.ones(i + 1, bool) if self.kinds[h] else (at < self.S) | (i - at < self.R)
        return attend(self.q[b][1][i, j], self.k[b][1][:i + 1, h][see], self.v[b][1][:i + 1, h][see])

    def check_rows(self, got, b, first, rows, what=""):
        """got: float64 [tokens, Hq, D] of positions first ...; rows: the ones to look at."""
        for t in rows:
            for j in range(self.Hq):
                ref, tol = self.expected(b, first + t, j)
                check(got[t, j], ref, tol, f"{what} sequence {b} position {first + t} head {j}")


def _some(rng, T, most):
    if T <= most:
        return range(T)
    return sorted({0, 1, T - 1, T - 2} | set(rng.integers(0, T, most).tolist()))


def _prefill(x, pad=0, most=6, **kw):
    from streaming_kv_cache_duo_gb300 import duo_device_error
    start, new = [n for n, _ in x.seqs], [T for _, T in x.seqs]
    q, k, v = (x.packed(y, start, new, pad) for y in (x.q, x.k, x.v))
    out = torch.full_like(q, 7.0)
    x.layer.prefill_ragged(q, k, v, x.map(start, new, pad), out=out, **kw)
    torch.cuda.synchronize()
    assert duo_device_error() == 0
    got = f64(out)
    at = 0
    for b, T in enumerate(new):
        x.check_rows(got[at:at + T], b, start[b], _some(x.rng, T, most), "prefill")
        assert np.isfinite(got[at:at + T]).all()
        at += T
    assert (got[at:] == 7).all()
    return out


CHUNKS = [
    # (cached, new) tokens, query heads, KV heads, retrieval heads, D, S, R, page
    ([(0, 1)], 1, 1, 1, 64, 4, 32, 128),
    ([(1, 1), (0, 2), (127, 1), (128, 1), (129, 3)], 4, 2, 1, 128, 4, 32, 128),
    ([(0, 300)], 4, 4, 2, 128, 64, 100, 128),
    ([(0, 17), (500, 33), (40, 0), (255, 128), (256, 129)], 8, 2, 1, 64, 3, 50, 256),
    ([(1000, 64), (3, 700), (0, 65)], 8, 1, 1, 128, 0, 20, 128),
    ([(777, 257), (0, 255), (30, 31)], 4, 4, 1, 64, 130, 7, 384),
    ([(2000, 1), (0, 1000), (900, 1), (5, 1), (1500, 600)], 16, 4, 2, 128, 64, 256, 128),
    ([(50, 400), (0, 90)], 6, 3, 0, 128, 16, 1, 128),   # no retrieval head, R = 1
    ([(300, 40), (1, 513)], 4, 2, 2, 128, 16, 64, 128),  # no streaming head
    ([(0, 40), (10, 30)], 2, 1, 0, 64, 500, 300, 128),   # sinks longer than all tokens
]


@pytest.mark.parametrize("case", CHUNKS, ids=[str(i) for i in range(len(CHUNKS))])
def test_chunks(case):
    _prefill(Batch(11, *case), pad=5)


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 4, 1), (64, 2, 2), (128, 8, 1)])
def test_items_shared_by_many_ctas(D, Hq, Hkv):
    """One sequence, few items: all CTAs share them; and one CTA's share ends inside an item."""
    _prefill(Batch(3, [(20000, 5)], Hq, Hkv, 1, D, 4, 32, 256), most=2)
    _prefill(Batch(4, [(9000, 333), (100, 1)], Hq, Hkv, 1, D, 4, 32, 128), most=2)


def test_many_sequences():
    """More sequences than a CTA has threads, some without a token."""
    rng = np.random.default_rng(8)
    seqs = [(int(rng.integers(0, 300)), int(rng.integers(0, 4))) for _ in range(900)]
    seqs[0], seqs[899], seqs[400] = (2000, 3), (1, 2), (700, 140)
    _prefill(Batch(9, seqs, 2, 2, 1, 64, 4, 32, 128), pad=3, most=1)


def test_streaming_heads_with_long_windows():
    _prefill(Batch(5, [(6000, 700), (10, 2500), (3000, 1)], 4, 2, 1, 128, 200, 2048, 128), most=4)
    _prefill(Batch(6, [(5000, 3)], 4, 2, 0, 64, 0, 4500, 128), most=3)


def test_sequences_turned_down_keep_their_rows():
    from streaming_kv_cache_duo_gb300 import duo_device_error
    x = Batch(7, [(100, 30), (50, 20), (0, 10)], 4, 2, 1, 64, 4, 32, 128)
    start, new = [100, None, 0], [30, 20, 10]
    q, k, v = (x.packed(y, start, new, 4) for y in (x.q, x.k, x.v))
    q[30:50] = k[30:50] = v[30:50] = NAN
    out = torch.full_like(q, 7.0)
    x.layer.prefill_ragged(q, k, v, x.map(start, new, 4), out=out)
    torch.cuda.synchronize()
    assert duo_device_error() == 0
    got = f64(out)
    assert (got[30:50] == 7).all() and (got[60:] == 7).all()
    x.check_rows(got[:30], 0, 100, range(0, 30, 7))
    x.check_rows(got[50:60], 2, 0, range(10))
    # a map whose last sequences do not fit in the packed batch at all
    m = x.map([100, None, None], [30, 20, 10])
    m.cu_new[2], m.cu_new[3] = 5000, 2 ** 31 - 1
    out.fill_(7.0)
    x.layer.prefill_ragged(q[:60], k[:60], v[:60], m, out=out[:60])
    torch.cuda.synchronize()
    assert duo_device_error() == 0 and (out[30:] == 7).all() and not (out[:30] == 7).any()


def _error(code_expected):
    from streaming_kv_cache_duo_gb300 import _lib
    code = ctypes.c_uint32()
    assert _lib.library().duo_device_error(ctypes.byref(code)) == code_expected


@pytest.mark.parametrize("bad", ["falls", "negative", "passes", "far", "capacity"])
def test_lengths_out_of_range_skip_their_sequence(bad):
    from streaming_kv_cache_duo_gb300 import _lib, duo_device_error
    x = Batch(7, [(100, 30), (50, 20), (0, 10)], 4, 2, 1, 64, 4, 32, 128)
    start, new = [100, 50, 0], [30, 20, 10]
    q, k, v = (x.packed(y, start, new) for y in (x.q, x.k, x.v))
    m = x.map(start, new)
    lost = [1]
    if bad == "falls":
        m.cu_new[2] = 20
        lost = [1, 2]  # (the third now begins at 20, inside the first, whose rows from there on it shares)
    elif bad == "negative":
        m.cu_new[0] = -3
        lost = [0]
    elif bad == "passes":
        m.cu_new[3] = 61
        lost = [2]
    elif bad == "far":
        m.token_pos[30] = 2 ** 31 - 20
    else:
        m.token_pos[30] = 129 * 1000
    out = torch.full_like(q, 7.0)
    x.layer.prefill_ragged(q, k, v, m, out=out)
    _error(_lib.DUO_ERR_INVALID_ARG)
    got = f64(out)
    at = [0, 30, 50, 60]
    for b in range(3):
        if b not in lost:
            x.check_rows(got[at[b]:at[b + 1]], b, start[b], [0, 19 if bad == "falls" else new[b] - 1])
    if bad != "falls":
        b = lost[0]
        assert (got[at[b]:at[b + 1]] == 7).all()
    assert duo_device_error() == 0


def _decode(x, max_len=None, most=None, **kw):
    from streaming_kv_cache_duo_gb300 import duo_device_error
    lens = [n + T for n, T in x.seqs]
    q = torch.stack([x.q[b][0][max(n - 1, 0)] if n else torch.full((x.Hq, x.D), NAN, dtype=torch.bfloat16)
                     for b, n in enumerate(lens)]).cuda()
    L = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = x.layer.decode_varlen(q, L, max_len or max(max(lens), 1), **kw)
    torch.cuda.synchronize()
    assert duo_device_error() == 0
    got = f64(out)
    assert np.isfinite(got).all()
    for b in _some(x.rng, x.B, most or x.B):
        if lens[b] == 0:
            assert (got[b] == 0).all()
        else:
            x.check_rows(got[b:b + 1], b, lens[b] - 1, [0], "decode")
    return out


DECODES = [
    ([1], 1, 1, 1, 64, 4, 32, 128),
    ([2, 0, 1, 127, 128, 129], 4, 2, 1, 128, 4, 32, 128),
    ([272, 300], 4, 4, 2, 64, 4, 32, 128),
    ([5000, 1, 0, 700, 257], 32, 4, 1, 128, 64, 256, 256),
    ([3000, 2999], 8, 8, 8, 64, 16, 64, 128),
    ([900, 20, 4000], 6, 3, 0, 128, 16, 1000, 128),
    ([15, 16, 17, 31, 33, 113], 2, 2, 1, 128, 0, 1, 384),
]


@pytest.mark.parametrize("case", DECODES, ids=[str(i) for i in range(len(DECODES))])
def test_single_tokens(case):
    lens, rest = case[0], case[1:]
    _decode(Batch(21, [(max(n - 1, 0), min(n, 1)) for n in lens], *rest, appended=True))


def test_single_tokens_of_many_sequences():
    rng = np.random.default_rng(2)
    lens = [int(n) for n in rng.integers(0, 400, 700)]
    lens[5] = 9000
    _decode(Batch(22, [(max(n - 1, 0), min(n, 1)) for n in lens], 4, 2, 1, 64, 4, 32, 128, appended=True), most=40)


def test_one_long_sequence():
    _decode(Batch(23, [(40000, 1)], 8, 2, 1, 128, 4, 32, 256, appended=True))


@pytest.mark.parametrize("D,Hq,Hkv,scale", [(64, 8, 1, 1.0), (64, 1, 1, 4.0), (128, 2, 1, 4.0)])
def test_long_sequences_shared_by_many_ctas(D, Hq, Hkv, scale):
    _decode(Batch(27, [(9000, 1), (0, 0), (20000, 1)], Hq, Hkv, Hkv, D, 4, 32, 128, appended=True, scale=scale))


@pytest.mark.parametrize("D,Hq", [(128, 8), (64, 4)])
def test_single_tokens_are_off_by_their_own_rounding(D, Hq):
    """P is a sum of two bf16 terms there, which leaves 2^-17 of it, sums are fp32: next to the outputs' rounding
    (some 2^-9.2 of their norm) that is nothing, and an eighth more is allowed. One term would be off by
    as much again, and the norm of both by 1.4 of the rounding's."""
    x = Batch(28, [(3000, 1), (1500, 1)], Hq, 1, 1, D, 4, 32, 128, appended=True)
    got = f64(_decode(x))
    ref = np.stack([np.stack([x.expected(b, n, j)[0] for j in range(Hq)]) for b, (n, _) in enumerate(x.seqs)])
    own = f64(torch.tensor(ref).to(torch.bfloat16)) - ref
    assert np.linalg.norm(got - ref) < 1.125 * np.linalg.norm(own)


@pytest.mark.parametrize("g", [1, 2, 4, 8])
def test_short_chunks_beside_long_ones(g):
    """Up to eight packed rows, and one more, in one call with more."""
    few = 8 // g
    x = Batch(29, [(700, few), (130, few + 1), (0, 300), (64, max(1, few - 1)), (1000, few)], g, 1, 1, 128, 4, 32, 128)
    _prefill(x, pad=3)


def test_lengths_past_max_len_are_clamped():
    """As if the caches held max_len tokens: the same outputs as those lengths give."""
    x = Batch(24, [(299, 1), (99, 1)], 4, 2, 2, 64, 4, 32, 128, appended=True)
    q = torch.stack([x.q[0][0][199], x.q[1][0][99]]).cuda()
    L = lambda *n: torch.tensor(n, dtype=torch.int32, device="cuda")
    a = x.layer.decode_varlen(q, L(300, 100), 200)
    b = x.layer.decode_varlen(q, L(200, 100), 200)
    c = x.layer.decode_varlen(q, L(200, -7), 200)
    assert torch.equal(a, b) and torch.equal(c[0], b[0]) and (c[1] == 0).all()


def test_chunk_of_single_tokens_equals_the_decode():
    """The same tokens as chunks of one before they are appended, and as single tokens after."""
    x = Batch(25, [(400, 1), (0, 1), (129, 1)], 8, 2, 1, 128, 4, 32, 128)
    _prefill(x)
    x.append([400, 0, 129], [1, 1, 1])
    _decode(x)


@pytest.mark.parametrize("scale", [4.0, 8.0])
def test_peaked_rows(scale):
    """Scores far apart: running maxima move many times."""
    _prefill(Batch(26, [(1500, 40), (0, 300)], 4, 2, 1, 128, 4, 64, 128, scale=scale), most=10)
    _decode(Batch(27, [(2999, 1), (200, 1)], 8, 2, 1, 64, 4, 64, 128, appended=True, scale=scale))


def test_infinities_behind_a_sequence_do_not_reach_it():
    """Other sequences' rows hold infinities: their own outputs are what they are, nobody else's change."""
    x = Batch(28, [(140, 21), (77, 50), (0, 9)], 4, 2, 1, 64, 4, 32, 128)
    start, new = [140, 77, 0], [21, 50, 9]
    q, k, v = (x.packed(y, start, new) for y in (x.q, x.k, x.v))
    m = x.map(start, new)
    a = x.layer.prefill_ragged(q, k, v, m)
    k[21:71], v[21:71] = float("inf"), float("-inf")
    b = x.layer.prefill_ragged(q, k, v, m)
    torch.cuda.synchronize()
    assert torch.equal(a[:21], b[:21]) and torch.equal(a[71:], b[71:]) and not torch.isfinite(b[21:71]).all()


@pytest.mark.parametrize("where", ["first", "middle", "last", "all"])
def test_bad_blocks_are_left_out(where):
    from streaming_kv_cache_duo_gb300 import _lib, duo_device_error
    x = Batch(29, [(700, 30), (300, 20)], 4, 2, 2, 64, 4, 32, 128)
    blocks = {"first": [0], "middle": [2], "last": [5], "all": range(6)}[where]
    for i in blocks:
        x.table[0, 1, i] = -1 if i % 2 else x.layer.k_full.shape[0]
    start, new = [700, 300], [30, 20]
    q, k, v = (x.packed(y, start, new) for y in (x.q, x.k, x.v))
    out = f64(x.layer.prefill_ragged(q, k, v, _map_of(x, start, new)))
    _error(_lib.DUO_ERR_INVALID_ARG)
    x.check_rows(out[30:], 1, 300, [0, 19])
    gone = np.concatenate([np.arange(i * 128, min(700, (i + 1) * 128)) for i in blocks])
    for t in (0, 29):
        for j in range(4):
            h = j // 2
            keep = np.ones(701 + t, bool)
            if h == 1:
                keep[gone] = False
            ref, tol = attend(x.q[0][1][700 + t, j], x.k[0][1][:701 + t, h][keep], x.v[0][1][:701 + t, h][keep])
            check(out[t, j], ref, tol, f"{t} {j}")
    if where == "all":  # a decode of it: nothing is left to see
        L = torch.tensor([700, 300], dtype=torch.int32, device="cuda")
        o = x.layer.decode_varlen(q[:2].contiguous(), L, 700)
        _error(_lib.DUO_ERR_INVALID_ARG)
        assert (o[0, 2:] == 0).all() and (o[0, :2] != 0).any()
    assert duo_device_error() == 0


def _map_of(x, start, new):
    """A slot map whose slots are not looked at (the table holds bad blocks)."""
    good = x.table.clone()
    x.table.clamp_(0, x.layer.k_full.shape[0] - 1)
    m = x.map(start, new)
    x.table.copy_(good)
    return m


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 4, 1), (64, 2, 2)])
def test_streaming_heads_at_the_last_positions(D, Hq, Hkv):
    """Chunks and single tokens up to position 2^31 - 2: what is 32-bit does not pass its range."""
    from streaming_kv_cache_duo_gb300 import DuoPagedLayer, duo_device_error
    rng, S, R, before = np.random.default_rng(37), 4, 40, 60
    for T in (9, 70, 300):
        first = 2 ** 31 - 1 - T
        k, v, q = (normal(rng, before + T, h, D) for h in (Hkv, Hkv, Hq))
        layer = DuoPagedLayer(1, Hq, Hkv, D, S, R, 128, 1, 1, None, [0] * Hkv)
        m = slot_map(None, 128, [first - before], [before])
        layer.append_ragged(k[0][:before].cuda(), v[0][:before].cuda(), m)
        m = slot_map(None, 128, [first], [T])
        qc, kc, vc = (x[0][before:].cuda() for x in (q, k, v))
        got = f64(layer.prefill_ragged(qc, kc, vc, m))
        layer.append_ragged(kc, vc, m)
        n = torch.tensor([2 ** 31 - 1], dtype=torch.int32, device="cuda")
        last = f64(layer.decode_varlen(qc[-1:], n, 2 ** 31 - 1))
        assert duo_device_error() == 0
        for t in range(T):
            i = before + t
            for j in range(Hq):
                see = slice(i - R + 1, i + 1)
                ref, tol = attend(q[1][i, j], k[1][see, j * Hkv // Hq], v[1][see, j * Hkv // Hq])
                check(got[t, j], ref, tol, f"chunk of {T}: {t}")
                if t == T - 1:
                    check(last[0, j], ref, tol, f"single token after {T}")


def test_calls_repeat_and_streams():
    """Equal results call after call (no order of atomics in them), on another stream, into a slice of rows."""
    x = Batch(30, [(3000, 60), (0, 200), (40, 1)], 8, 2, 1, 128, 4, 32, 128)
    start, new = [3000, 0, 40], [60, 200, 1]
    q, k, v = (x.packed(y, start, new) for y in (x.q, x.k, x.v))
    m = x.map(start, new)
    a = x.layer.prefill_ragged(q, k, v, m)
    for _ in range(3):
        assert torch.equal(x.layer.prefill_ragged(q, k, v, m), a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = torch.empty_like(a)
    x.layer.prefill_ragged(q, k, v, m, out=b, stream=s)
    s.synchronize()
    assert torch.equal(a, b)
    fused = torch.cat([q, k, v], 1)  # slices of a projection's output
    qs, ks, vs = fused.split([8, 2, 2], 1)
    assert torch.equal(x.layer.prefill_ragged(qs, ks, vs, m), a)


def test_captured_step_replays_with_other_lengths():
    """Tables, rotation, append and decode of single tokens in one CUDA graph, lengths on the device."""
    from streaming_kv_cache_duo_gb300 import DuoBlockPool, DuoPagedLayer, DuoRope, duo_device_error
    from ragged_util import rotated
    rng = np.random.default_rng(31)
    B, Hq, Hkv, D, S, R, page, steps = 3, 8, 2, 128, 4, 32, 128, 6
    kinds = [1, 0]
    pool = DuoBlockPool(B, 1, page, 4, 16, 600)
    layer = DuoPagedLayer(B, Hq, Hkv, D, S, R, page, 4, 16, pool.block_table, kinds)
    rope = DuoRope(D, scaling=dict(kind="yarn", factor=4.0, original=64))
    lens = [130, 0, 126]
    total = [n + steps for n in lens]
    qkv = [normal(rng, t, Hq + 2 * Hkv, D) for t in total]
    # chunks first: rotate, attend, append
    first = DuoBlockPool.update(pool, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    x = torch.cat([qkv[b][0][:lens[b]] for b in range(B)]).cuda()
    x = torch.cat([x, torch.full((600 - len(x),) + tuple(x.shape[1:]), NAN, dtype=torch.bfloat16, device="cuda")])
    q, k, v = x.split([Hq, Hkv, Hkv], 1)
    qr, kr = rope.rotate(q, k, first.token_pos)
    chunk = layer.prefill_ragged(qr, kr, v, first)
    layer.append_ragged(kr, v, first)
    torch.cuda.synchronize()
    assert duo_device_error() == 0

    def expected(b, i):
        y, _ = rotated(qkv[b][1][:i + 1], np.arange(i + 1), rope.inv_freq, D, "half", rope.scale)
        bf = lambda t: torch.tensor(t).to(torch.bfloat16).double().numpy()
        qy, ky, vy = bf(y[i, :Hq]), bf(y[:, Hq:Hq + Hkv]), qkv[b][1][:i + 1, Hq + Hkv:]
        out, tol = np.zeros((Hq, D)), np.zeros((Hq, D))
        for j in range(Hq):
            h, at = j // (Hq // Hkv), np.arange(i + 1)
            see = np.ones(i + 1, bool) if kinds[h] else (at < S) | (i - at < R)
            # (q and k: where fp32 and 64 bits round to different bf16 values, they are a step of 2^-7 apart)
            out[j], tol[j] = attend(qy[j], ky[see, h], vy[see, h], kv_rounding=2.0 ** -7)
        return out, tol

    got, at = f64(chunk), 0
    for b in range(B):
        for t in sorted({0, lens[b] - 1} if lens[b] else ()):
            check(got[at + t], *expected(b, t), f"chunk {b} {t}")
        at += lens[b]
    # single tokens: one graph, replayed
    step_pool = DuoBlockPool(B, 1, page, 4, 16, B)
    for name in ("block_table", "free_list", "free_count", "seq_lens"):
        getattr(step_pool, name).copy_(getattr(pool, name))
    layer.block_table.copy_(step_pool.block_table)
    layer2_table = step_pool.block_table
    layer.paged.block_table = layer2_table.data_ptr()
    new = torch.ones(B, dtype=torch.int32, device="cuda")
    x = torch.zeros(B, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device="cuda")
    q, k, v = x.split([Hq, Hkv, Hkv], 1)
    qr, out = torch.empty(B, Hq, D, dtype=torch.bfloat16, device="cuda"), torch.empty(B, Hq, D, dtype=torch.bfloat16, device="cuda")

    def step():
        m = step_pool.update(new)
        layer.append_ragged(k, v, m, rope=rope, q=q, q_out=qr)
        layer.decode_varlen(qr, step_pool.seq_lens, 4 * page, out=out)

    graph = torch.cuda.CUDAGraph()
    for s in range(steps):
        x.copy_(torch.stack([qkv[b][0][lens[b] + s] for b in range(B)]))
        if s == 0:
            step()
        else:
            if s == 1:
                with torch.cuda.graph(graph):
                    step()
            graph.replay()
        torch.cuda.synchronize()
        assert duo_device_error() == 0
        for b in range(B):
            check(f64(out)[b], *expected(b, lens[b] + s), f"step {s} sequence {b}")


def test_refusals():
    from streaming_kv_cache_duo_gb300 import DuoError, _lib
    x = Batch(33, [(10, 3), (0, 4)], 4, 2, 1, 64, 4, 32, 128)
    L, m = x.layer, x.map([10, 0], [3, 4])
    q, k, v = (x.packed(y, [10, 0], [3, 4]) for y in (x.q, x.k, x.v))
    lens = torch.tensor([10, 0], dtype=torch.int32, device="cuda")
    for call in (lambda: L.prefill_ragged(q[:6], k, v, m), lambda: L.prefill_ragged(q, k[:, :1], v, m),
                 lambda: L.prefill_ragged(q, k, v.float(), m), lambda: L.prefill_ragged(q, k, v, m, out=q[:, :2]),
                 lambda: L.prefill_ragged(q, k, v, x.map([10], [7])), lambda: L.decode_varlen(q, lens, 100),
                 lambda: L.decode_varlen(q[:2], lens.cpu(), 100), lambda: L.decode_varlen(q[:2], lens[:1], 100),
                 lambda: L.decode_varlen(q[:2].transpose(0, 1), lens, 100)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(DuoError, match="DUO_ERR_INVALID_ARG"):
        L.decode_varlen(q[:2], lens, 0)
    with pytest.raises(DuoError, match="DUO_ERR_INVALID_ARG"):
        L.decode_varlen(q[:2], lens, 129)  # past the tables
    for call in (lambda: L.prefill_ragged(q, k, v, m, out=q), lambda: L.decode_varlen(q[:2], lens, 100, out=q[:2])):
        with pytest.raises(DuoError, match="DUO_ERR_INVALID_ARG"):
            call()
    with pytest.raises(NotImplementedError):
        L.append_varlen(k, v, lens)
    o, need = torch.empty_like(q), _lib.duo_prefill_ragged_workspace_size(L.handle, 7)
    ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    with pytest.raises(DuoError, match="DUO_ERR_WORKSPACE"):
        _lib.duo_attn_prefill_ragged(L.handle, L.cache, L.paged, m.c, 7, q, k, v, o, ws[:need - 1])
    with pytest.raises(DuoError, match="DUO_ERR_INVALID_ARG"):
        _lib.duo_attn_prefill_ragged(L.handle, L.cache, L.paged, m.c, 7, q, k, v, o, ws[8:])
    with pytest.raises(DuoError, match="DUO_ERR_WORKSPACE"):
        _lib.duo_attn_decode_paged_varlen(L.handle, L.cache, L.paged, lens, 100, q[:2], o[:2], None)
    _lib.duo_attn_prefill_ragged(L.handle, L.cache, L.paged, m.c, 7, q, k, v, o, ws[:need])
    e = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert L.prefill_ragged(e, e[:, :2], e[:, :2], x.map([10, 0], [0, 0])).shape[0] == 0
    L.paged.stream_table = L.paged.block_table
    with pytest.raises(DuoError, match="DUO_ERR_UNSUPPORTED"):
        L.decode_varlen(q[:2], lens, 100)
