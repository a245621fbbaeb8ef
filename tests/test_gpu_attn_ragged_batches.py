"""Packed attention over batches of the sizes where the way a CTA finds its share of the work changes: one warp
sums up to 32 sequences, all threads one sequence each up to 384, and more in rounds. Empty sequences stand at
both ends, and a long one, whose tiles many CTAs share, in the last place."""

import numpy as np
import pytest

from test_gpu_attn_ragged import Batch, _decode, _prefill

pytestmark = pytest.mark.gpu
SIZES = [31, 32, 33, 48, 64, 128, 383, 384, 385]


def _lengths(B, most):
    rng = np.random.default_rng(B)
    n = [int(x) for x in rng.integers(0, most, B)]
    n[-1] = 6000
    return rng, n


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 2, 2), (128, 8, 2)])
@pytest.mark.parametrize("B", SIZES)
def test_single_tokens(B, D, Hq, Hkv):
    _, n = _lengths(B, 400)
    n[0] = n[1] = n[-2] = 0
    _decode(Batch(61, [(max(x - 1, 0), min(x, 1)) for x in n], Hq, Hkv, 1, D, 4, 32, 128, appended=True), most=30)


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 2, 2), (128, 8, 2)])
@pytest.mark.parametrize("B", SIZES)
def test_chunks(B, D, Hq, Hkv):
    rng, n = _lengths(B, 300)
    new = [int(x) for x in rng.integers(0, 4, B)]
    new[0] = new[1] = new[-2] = 0
    new[-1], new[B // 2] = 5, 150
    x = Batch(62, list(zip(n, new)), Hq, Hkv, 1, D, 4, 32, 128)
    _prefill(x, pad=3, most=1 if B > 64 else 2)


@pytest.mark.parametrize("B", [32, 33, 384, 385])
def test_the_last_sequence_is_the_only_one(B):
    """All but it are empty, or turned down: every CTA's share is in the last sequence."""
    n = [0] * (B - 1) + [3000]
    _decode(Batch(63, [(max(x - 1, 0), min(x, 1)) for x in n], 2, 2, 1, 64, 4, 32, 128, appended=True), most=3)
    _prefill(Batch(64, [(0, 0)] * (B - 1) + [(900, 200)], 2, 2, 1, 64, 4, 32, 128), pad=2, most=3)


@pytest.mark.parametrize("B", [1, 32, 33, 385])
def test_no_sequence_holds_anything(B):
    """No work at all: zeros from single tokens, nothing written by chunks."""
    import torch
    from streaming_kv_cache_duo_gb300 import duo_device_error
    x = Batch(65, [(0, 0)] * B, 4, 2, 1, 64, 4, 32, 128)
    q = torch.randn(B, 4, 64, device="cuda").to(torch.bfloat16)
    out = torch.full_like(q, 7.0)
    x.layer.decode_varlen(q, torch.zeros(B, dtype=torch.int32, device="cuda"), 100, out=out)
    assert (out == 0).all()
    pad = 6
    q, k, v = (torch.full((pad, h, 64), float("nan"), dtype=torch.bfloat16, device="cuda") for h in (4, 2, 2))
    out = torch.full_like(q, 7.0)
    x.layer.prefill_ragged(q, k, v, x.map([None] * B, [0] * B, pad), out=out)
    assert (out == 7).all() and duo_device_error() == 0
