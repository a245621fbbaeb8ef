"""Helpers of the packed-step tests: slot maps, rotations and attention in 64 bits, with bounds."""

from __future__ import annotations

import numpy as np

from kv8_util import BF16, FP32, bf16, f64, normal, scattered_table, slot_of  # noqa: F401


def kinds_of(Hkv, n_ret):
    """n_ret of Hkv heads, spread."""
    return [1 if (h * n_ret) // Hkv != ((h + 1) * n_ret) // Hkv else 0 for h in range(Hkv)]


def slot_map(table, page, start, new, pad=0, planes=None):
    """DuoSlotMap of sequences that take new[b] tokens after start[b] (None: turned down), `pad` tokens of
    padding behind them. table: int32 CUDA [B, planes, max_blocks], or None without retrieval heads."""
    import torch
    from streaming_kv_cache_duo_gb300 import DuoSlotMap
    seq, pos, cu = [], [], [0]
    for b, n in enumerate(new):
        seq += [b] * n
        pos += [-1] * n if start[b] is None else list(range(start[b], start[b] + n))
        cu.append(cu[-1] + n)
    seq += [-1] * pad
    pos += [-1] * pad
    N = len(seq)
    planes = 0 if table is None else table.shape[1]
    slots = np.full((N, planes), -1, np.int64)
    if planes:
        t = table.cpu().numpy()
        for i in range(N):
            if pos[i] >= 0:
                slots[i] = t[seq[i], :, pos[i] // page].astype(np.int64) * page + pos[i] % page
    dev = lambda x, d: torch.tensor(np.asarray(x), dtype=d).cuda()
    return DuoSlotMap(dev(cu, torch.int32), dev(seq, torch.int32), dev(pos, torch.int32),
                      dev(slots, torch.int64).reshape(N, planes))


def rotated(x, pos, freq, rotary, layout, scale=1.0):
    """Rows x [N, heads, D] (float64) turned by the tokens' positions, and a bound on a kernel's error.

    The bound: the angle as a number of half turns is rounded to fp32 (2^-24 of at most 1, after 2^-31 for
    the bits left out), so off by pi (2^-24 + 2^-31) rad; sin and cos of it are good to two units in the last
    place (2^-23 each), scaled with one more rounding; two products and a sum round three times at 2^-24:
    (|a| + |b|) scale times pi 2^-24 + 2^-22 + 4 2^-24 < 2^-20 in all. The 64-bit reference's own angle is
    off by 2^-53 of its size. The result is rounded to bf16 once (2^-8 of it)."""
    y = x.copy()
    tol = np.zeros_like(x)
    half = rotary // 2
    a = np.arange(half) if layout == "half" else 2 * np.arange(half)
    b = a + half if layout == "half" else a + 1
    angle = np.asarray(pos, np.float64)[:, None, None] * np.asarray(freq)
    c, s = np.cos(angle) * scale, np.sin(angle) * scale
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    size = scale * (np.abs(x[..., a]) + np.abs(x[..., b]))
    d = size * (2.0 ** -20 + np.abs(angle) * 2.0 ** -52)
    tol[..., a] = BF16 * (np.abs(y[..., a]) + d) + d
    tol[..., b] = BF16 * (np.abs(y[..., b]) + d) + d
    return y, tol
