"""Helpers of the 8-bit cache tests: expected caches, attention in 64 bits with a bound on the
error of every output, and reading the device's arrays."""

from __future__ import annotations

import numpy as np

from oracle.kv8 import BLOCK, Kv8Rows

BF16 = 2.0 ** -8   # half a step of a bf16 rounding, relative to the value
FP16 = 2.0 ** -11
FP32 = 2.0 ** -24


def bf16(x):
    """float array -> (bf16 CPU tensor, float64 array of exactly its values)."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)
    return t, t.to(torch.float64).numpy()


def normal(rng, *shape, scale=1.0):
    return bf16(rng.standard_normal(shape) * scale)


def f64(t):
    """Device tensor of any type -> float64 values."""
    return t.float().cpu().numpy().astype(np.float64)


def expected_rows(k, code, splits=None):
    """Kv8Rows of one head's rows k [n, D]."""
    r = Kv8Rows(k.shape[1], code)
    at = 0
    for n in splits or [len(k)]:
        r.append(k[at:at + n])
        at += n
    return r


def slot_of(t, S, R):
    return t if t < S else S + (t - S) % R


def ring(rows, S, R):
    """What a sink + ring cache holds after rows [n, D]: (positions [S + R], rows [S + R, D])."""
    pos = np.full(S + R, -1)
    out = np.zeros((S + R, rows.shape[1]))
    for t in range(len(rows)):
        pos[slot_of(t, S, R)] = t
        out[slot_of(t, S, R)] = rows[t]
    return pos, out


def attend(q, k, v, n_codes=0, kv_rounding=0.0):
    """softmax(q k / sqrt D) v of one query over the keys it sees, in 64 bits, and a bound on
    what a kernel may be off by, element for element. k, v [keys, D]: the values the cache
    stands for; the first n_codes of them are held in codes.

    The bound: the output's rounding to bf16 (2^-8 |o|); p rounded to fp16 over codes and to
    bf16 over bf16 rows while the sum of p is not, so |dp| <= u p with u = 2^-11 or 2^-8; each
    score off by ds <= (D + 4) 2^-23 sum |q||k| / sqrt D (fp32 sums of exact products, twice
    2^-24 a step as tensor-core sums may truncate), which turns p into p e^(+-ds) in numerator
    and denominator: 2 ds; fp32 sums of p v: (keys per warp and lane, at most 2^10 steps here)
    2^-13 of sum p |v| at the very worst, ex2.approx 2^-22, p's flush below 2^-31 of the
    maximum (keys 2^-31). kv_rounding: relative rounding of k and v before the products."""
    D = q.shape[-1]
    if len(k) == 0:
        return np.zeros(D), np.zeros(D)
    s = k @ q / np.sqrt(D)
    mass = np.abs(k) @ np.abs(q) / np.sqrt(D)
    ds = (D + 4) * 2 * FP32 * mass.max() + 4 * FP32 * np.abs(s).max() + kv_rounding * mass.max()
    p = np.exp(s - s.max())
    l = p.sum()
    o = p @ v / l
    u = np.where(np.arange(len(k)) < n_codes, FP16, BF16)
    av = np.abs(v)
    spread = (p * (u + kv_rounding + 2.0 ** -13 + 2.0 ** -21)) @ av / l + 2 * np.expm1(ds) * (p @ av) / l
    spread += len(k) * 2.0 ** -31 * av.max(0)
    return o, BF16 * (np.abs(o) + spread) + spread


def check(got, ref, tol, what=""):
    got = np.asarray(got, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    worst = np.max(np.abs(got - ref) - tol)
    assert worst <= 0, f"{what}: {worst:.3e} past the bound; max err {np.abs(got - ref).max():.3e}"


class Batch:
    """A batch of sequences of given lengths: bf16 q, k, v per position, and what every head's
    cache holds of each."""

    def __init__(self, seed, lens, Hq, Hkv, D, S, R, kinds, code, scale=1.0, room=0):
        rng = np.random.default_rng(seed)
        self.lens, self.kinds, self.code, self.D, self.S, self.R = list(lens), kinds, code, D, S, R
        self.Hq, self.Hkv, self.g, self.B = Hq, Hkv, Hq // Hkv, len(lens)
        self.ret = [h for h in range(Hkv) if kinds[h]]
        self.str_ = [h for h in range(Hkv) if not kinds[h]]
        self.L = max(max(lens) + room, 1)
        self.kt, self.k = normal(rng, self.B, self.L, Hkv, D, scale=scale)
        self.vt, self.v = normal(rng, self.B, self.L, Hkv, D)
        self.qt, self.q = normal(rng, self.B, self.L, Hq, D)

    def heads_rows(self, b, h, n, x):
        """Rows [0, n) of head h as a query sees them in the cache: (positions, values, full)."""
        rows = x[b, :n, h]
        if self.kinds[h]:
            return np.arange(n), expected_rows(rows, self.code).rows(), n // BLOCK * BLOCK
        return np.arange(n), rows, 0

    def decode(self, b, n):
        """Outputs [Hq, D] and bounds of the query at position n - 1 after n tokens."""
        out, tol = np.zeros((self.Hq, self.D)), np.zeros((self.Hq, self.D))
        if n == 0:
            return out, tol
        for h in range(self.Hkv):
            at, k, full = self.heads_rows(b, h, n, self.k)
            _, v, _ = self.heads_rows(b, h, n, self.v)
            see = np.ones(n, bool) if self.kinds[h] else (at < self.S) | (n - 1 - at < self.R)
            for j in range(h * self.g, (h + 1) * self.g):
                out[j], tol[j] = attend(self.q[b, n - 1, j], k[see], v[see], full)
        return out, tol

    def fill(self, layer, chunk=None):
        """Append the whole batch (equal lengths) to a layer."""
        n = self.lens[0]
        assert all(x == n for x in self.lens)
        step = chunk or n
        for t in range(0, n, step):
            e = min(n, t + step)
            layer.append(self.kt[:, t:e].contiguous().cuda(), self.vt[:, t:e].contiguous().cuda())

    def packed(self, start, new):
        """k, v of tokens start[b] ... start[b] + new[b] - 1 of every sequence, packed."""
        import torch
        pick = lambda x: torch.cat([x[b, start[b]:start[b] + new[b]] for b in range(self.B)]).contiguous().cuda()
        return pick(self.kt), pick(self.vt)

    def query(self, lens):
        """q [B, Hq, D] of each sequence's last token (any row for an empty one)."""
        import torch
        return torch.stack([self.qt[b, max(n - 1, 0)] for b, n in enumerate(lens)]).contiguous().cuda()


def scattered_table(rng, B, planes, max_blocks, extra=3):
    """int32 CUDA table [B, planes, max_blocks] of distinct blocks in a random order, and the pool's size."""
    import torch
    ids = rng.permutation(B * planes * max_blocks + extra)[:B * planes * max_blocks]
    return torch.from_numpy(ids.reshape(B, planes, max_blocks).astype(np.int32)).cuda(), B * planes * max_blocks + extra
