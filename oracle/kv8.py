"""8-bit cache blocks and block tables, restated in plain NumPy.

Blocks: 64 rows of one head share a scale, fp32(amax / 127) for int8 codes and fp32(amax /
448) for e4m3 ones; code = the quotient fp32(x / scale) rounded to nearest even on the code
grid and clamped to it. A block of zeros has scale 0 and codes 0, a block with a non-finite
value scale NaN and codes 0. Rows of the block that is not full stay as they are.

Block tables: the update of a step as a sequential program, request by request.
"""

from __future__ import annotations

import numpy as np

BLOCK = 64
TOP = {"int8": 127.0, "e4m3": 448.0}


def round_e4m3(x):
    """float64 array -> nearest e4m3 value (ties to even mantissa), saturating at +-448. The
    grid: 8 steps per power of two from 2^-6 up, and multiples of 2^-9 below."""
    x = np.asarray(x, np.float64)
    mag = np.minimum(np.abs(x), 448.0)
    e = np.floor(np.log2(np.maximum(mag, 2.0 ** -6)))
    # log2 may land on the wrong side of a power of two by rounding: put it right exactly
    e = np.where(np.exp2(e) > np.maximum(mag, 2.0 ** -6), e - 1, e)
    step = np.exp2(e - 3)
    return np.copysign(np.minimum(np.rint(mag / step) * step, 448.0), x)


def quantize_block(x, code):
    """[64, D] values (exactly representable in fp32) -> (code values float64 [64, D], fp32 scale)."""
    x = np.asarray(x, np.float32)
    if not np.isfinite(x).all():
        return np.zeros(x.shape), np.float32(np.nan)
    scale = np.float32(np.abs(x).max()) / np.float32(TOP[code])
    if scale == 0:
        return np.zeros(x.shape), np.float32(0)
    q = (x / scale).astype(np.float64)  # fp32 quotients
    c = np.rint(q) if code == "int8" else round_e4m3(q)
    return np.clip(c, -TOP[code], TOP[code]), scale


class Kv8Rows:
    """The rows of one (sequence, head), appended in any split."""

    def __init__(self, D, code):
        self.D, self.code = D, code
        self.codes, self.scales = [], []
        self.tail = np.zeros((0, D))

    def append(self, rows):
        self.tail = np.concatenate([self.tail, np.asarray(rows, np.float64)])
        while len(self.tail) >= BLOCK:
            c, s = quantize_block(self.tail[:BLOCK], self.code)
            self.codes.append(c)
            self.scales.append(s)
            self.tail = self.tail[BLOCK:]

    def rows(self):
        """float64 [n, D] the cache stands for."""
        with np.errstate(invalid="ignore"):
            full = [c * np.float64(s) for c, s in zip(self.codes, self.scales)]
        return np.concatenate(full + [self.tail]) if full else self.tail


def block_tables_update(table, free, count, lens, new, block_size, max_tokens):
    """One step on copies of the inputs. table int [B, planes, max_blocks], free int
    [num_blocks] with its first `count` entries free. Returns a dict of the results, and
    whether any sequence was turned down."""
    table, free, lens = table.copy(), list(free), list(int(v) for v in lens)
    B, planes, max_blocks = table.shape
    held = [-(-n // block_size) for n in lens]
    old = list(lens)
    count = int(count)
    for b in range(B):
        if new[b] == -1:
            for p in range(planes):
                for j in range(held[b]):
                    if 0 <= table[b, p, j] < len(free):  # an id that is none is dropped
                        free[count] = int(table[b, p, j])
                        count += 1
            lens[b] = 0
    cu = np.zeros(B + 1, np.int64)
    for b in range(B):
        cu[b + 1] = cu[b] + max(int(new[b]), 0)
    served, starved, turned_down = [False] * B, False, False
    for b in range(B):
        if new[b] < 0:
            continue
        fits = old[b] + new[b] <= max_blocks * block_size and (new[b] == 0 or cu[b + 1] <= max_tokens)
        want = planes * (-(-(old[b] + int(new[b])) // block_size) - held[b]) if fits else 0
        if fits and want and (starved or want > count):
            starved, fits = True, False
        if not fits:
            turned_down = True
            continue
        served[b] = True
        lens[b] = old[b] + int(new[b])
        for p in range(planes):
            for j in range(held[b], held[b] + want // planes):
                count -= 1
                table[b, p, j] = free[count]
    seq = np.full(max_tokens, -1)
    pos = np.full(max_tokens, -1)
    slots = np.full((max_tokens, planes), -1, np.int64)
    for b in range(B):
        for k in range(max(int(new[b]), 0)):
            i = cu[b] + k
            if i >= max_tokens:
                break
            seq[i] = b
            if served[b]:
                pos[i] = old[b] + k
                for p in range(planes):
                    slots[i, p] = int(table[b, p, pos[i] // block_size]) * block_size + pos[i] % block_size
    return dict(block_table=table, free_list=np.array(free), free_count=count, seq_lens=np.array(lens), cu_new=cu,
                token_seq=seq, token_pos=pos, slots=slots, turned_down=turned_down)
