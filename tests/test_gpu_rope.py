"""Rotary positions against the formula in 64 bits: layouts, part of the head, scaled frequencies, far
positions, strided and in-place rows, skipped tokens."""

import math

import numpy as np
import pytest
import torch

from kv8_util import check
from ragged_util import f64, normal, rotated

pytestmark = pytest.mark.gpu

SCALINGS = [None, dict(kind="linear", factor=4.0), dict(kind="ntk", factor=2.5),
            dict(kind="yarn", factor=8.0, original=4096),
            dict(kind="wavelength", factor=8.0, low=1.0, high=4.0, original=8192)]


def _positions(rng, N, far):
    pos = rng.integers(0, far, N)
    pos[0] = far - 1
    return pos


@pytest.mark.parametrize("N,Hq,Hkv,D,rd,layout,far", [
    (1, 4, 4, 64, 64, "half", 1), (1, 32, 8, 128, 128, "half", 2 ** 31 - 1), (7, 5, 1, 64, 16, "interleaved", 100),
    (64, 32, 8, 128, 128, "interleaved", 1 << 20), (333, 3, 2, 128, 48, "half", 5000), (33, 2, 2, 128, 96, "interleaved", 300000),
    (2500, 8, 4, 64, 48, "half", 1 << 24), (10001, 16, 2, 128, 64, "half", 131072),
])
def test_rotation(N, Hq, Hkv, D, rd, layout, far):
    from streaming_kv_cache_duo_gb300 import DuoRope
    rng = np.random.default_rng(N * 31 + rd)
    for scaling in SCALINGS if N < 400 else [SCALINGS[N % 5]]:
        rope = DuoRope(D, theta=50000.0, rotary_dim=rd, layout=layout, scaling=scaling)
        pos = _positions(rng, N, far)
        qt, q = normal(rng, N, Hq, D, scale=2.0)
        kt, k = normal(rng, N, Hkv, D)
        p = torch.tensor(pos, dtype=torch.int32).cuda()
        qo, ko = rope.rotate(qt.cuda(), kt.cuda(), p)
        for got, x in ((qo, q), (ko, k)):
            ref, tol = rotated(x, pos, rope.inv_freq, rd, layout, rope.scale)
            check(f64(got), ref, tol, f"{scaling}")
        assert torch.equal(qo[..., rd:].cpu(), qt[..., rd:])
    # the same in place, q alone
    x = qt.cuda()
    out, none = rope.rotate(x, None, p, q_out=x)
    assert none is None and out is x and torch.equal(x, qo)


def test_slices_and_skipped_tokens():
    """Slices of a fused projection in, slices of another tensor out; tokens at position -1 keep their rows."""
    from streaming_kv_cache_duo_gb300 import DuoRope
    rng = np.random.default_rng(5)
    N, Hq, Hkv, D = 50, 6, 2, 64
    rope = DuoRope(D)
    xt, x = normal(rng, N, Hq + 2 * Hkv, D)
    pos = rng.integers(-1, 40, N)
    pos[[0, N - 1]] = -1
    out = torch.full((N, Hq + Hkv + 3, D), 7.0, dtype=torch.bfloat16, device="cuda")
    q, k, _ = xt.cuda().split([Hq, Hkv, Hkv], 1)
    rope.rotate(q, k, torch.tensor(pos, dtype=torch.int32).cuda(), q_out=out[:, 1:1 + Hq], k_out=out[:, 2 + Hq:2 + Hq + Hkv])
    got = f64(out)
    real = pos >= 0
    ref, tol = rotated(x[real], pos[real], rope.inv_freq, D, "half")
    check(got[real][:, 1:1 + Hq], ref[:, :Hq], tol[:, :Hq])
    check(got[real][:, 2 + Hq:2 + Hq + Hkv], ref[:, Hq:Hq + Hkv], tol[:, Hq:Hq + Hkv])
    assert (got[~real] == 7).all() and (got[:, [0, 1 + Hq, 2 + Hq + Hkv]] == 7).all()


def test_far_angles_are_exact():
    """At positions up to 2^31 - 1, against the angle reduced with whole numbers: frequencies that are
    fractions of a turn with small denominators."""
    from streaming_kv_cache_duo_gb300 import DuoRope
    D, den = 64, [3, 5, 7, 11, 13, 17, 19, 23] * 4
    rope = DuoRope(D, inv_freq=[2 * math.pi / d for d in den])
    pos = np.array([0, 1, 22, 10 ** 6 + 3, 2 ** 30 + 7, 2 ** 31 - 2, 2 ** 31 - 1])
    x = torch.zeros(len(pos), 1, D, dtype=torch.bfloat16, device="cuda")
    x[..., :D // 2] = 1.0
    got = f64(rope.rotate(x, None, torch.tensor(pos, dtype=torch.int32).cuda())[0])[:, 0]
    for i, p in enumerate(pos.tolist()):
        for j, d in enumerate(den):
            t = 2 * math.pi * (p % d) / d
            # the frequency itself is a double: off by at most 2^-53 of it, times the position
            slack = 2.0 ** -20 + p * (2 * math.pi / d) * 2.0 ** -52
            assert abs(got[i, j] - math.cos(t)) <= 2.0 ** -8 * abs(math.cos(t)) + 2 * slack
            assert abs(got[i, j + D // 2] - math.sin(t)) <= 2.0 ** -8 * abs(math.sin(t)) + 2 * slack


def test_rotation_captured_and_on_another_stream():
    from streaming_kv_cache_duo_gb300 import DuoRope
    rng = np.random.default_rng(9)
    rope = DuoRope(128, layout="interleaved")
    qt, q = normal(rng, 40, 4, 128)
    x, out = qt.cuda(), torch.empty(40, 4, 128, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        rope.rotate(x, None, pos, q_out=out)
    s.synchronize()
    first = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rope.rotate(x, None, pos, q_out=out)
    for shift in (0, 1000):
        pos += shift
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        ref, tol = rotated(q, pos.cpu().numpy(), rope.inv_freq, 128, "interleaved")
        check(f64(out), ref, tol)
        if shift == 0:
            assert torch.equal(out, first)


def test_refusals():
    from streaming_kv_cache_duo_gb300 import DuoRope
    rope = DuoRope(64)
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    p = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (lambda: rope.rotate(q.half(), None, p), lambda: rope.rotate(q, None, p.long()),
                lambda: rope.rotate(q, None, p.cpu()), lambda: rope.rotate(q[:3], None, p),
                lambda: rope.rotate(q.transpose(1, 2), None, p), lambda: rope.rotate(q, q[..., :32], p),
                lambda: rope.rotate(q, None, p, q_out=q[:2]), lambda: rope.rotate(q.cpu(), None, p),
                lambda: rope.rotate(q[:1].expand(4, 2, 64), None, p)):
        with pytest.raises(ValueError):
            bad()
    out, _ = rope.rotate(q[:0], None, p[:0])  # no token
    assert out.shape[0] == 0
